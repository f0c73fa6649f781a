// conv_varlen.hip -- the causal depthwise conv over packed token-major rows
// (causal_conv1d_varlen_fwd) and its gradient (causal_conv1d_varlen_bwd).
//
// Both stream: the forward reads and writes every element once (4 bytes an
// element in 16 bits), the backward reads two and writes one.  A wave owns 64
// runs of NV neighbouring channels (16 bytes each where the rows allow it, so
// a token's load is one KiB) and walks a run of tokens with the last inputs in
// registers.  The three tokens before a run are read again.  85 us and 126 us at
// 16384 x 5376 bf16 are 4.2 TB/s of what they have to move.
// What a token may see is decided by wave-uniform scalars: its place in its
// sequence, found once per run in cu_seqlens and then counted.  The run's loads
// are issued together before the first is used.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "conv_runs.h"
#include "device_util.h"
#include "host_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kW = SSM_CONV_WIDTH;
static_assert(kW == kTaps, "one width");
constexpr int kFwdRun = 12;        // tokens of a wave's run, forward
constexpr int kBwdRun = 32;        // tokens of a wave's run, backward
constexpr int kShortRun = 4;       // the same where the waves are few, forward
constexpr int kShortBwdRun = 8;    // and backward
constexpr int kBwdVec = 4;        // channels of a lane, backward, 16 bits
constexpr int kStep = 4;           // tokens whose loads are in flight together, backward
constexpr int kRows = 4;           // waves (runs) of a workgroup

// NV neighbouring io elements (NV = 1: any alignment)
template <int IO, int NV>
struct Vec {
  RawV<IO, NV> r;
  __device__ __forceinline__ void load(const void *p, int64_t i) { r.load_vec(p, i); }
  __device__ __forceinline__ float get(int k) const { return r.get(k); }
  __device__ __forceinline__ void zero() { r.zero(); }
};
template <int IO>
struct Vec<IO, 1> {
  float v;
  __device__ __forceinline__ void load(const void *p, int64_t i) { v = load_io<IO>(p, i); }
  __device__ __forceinline__ float get(int) const { return v; }
  __device__ __forceinline__ void zero() { v = 0.0f; }
};
template <int IO, int NV>
__device__ __forceinline__ void put(void *p, int64_t i, const float (&v)[NV]) {
  if constexpr (NV == 1) store_one<IO>(p, i, v[0]);
  else store_n<IO, NV>(p, i, v, NV, true);
}

struct ConvVarParams {
  const void *x, *dout;
  void *out, *dx, *ring;
  const float *w, *bias;
  const int32_t *cu, *seen, *slots;
  float *part;                       // backward: (blocks of runs, kW + 1, channels)
  int64_t total, nseq, channels, xs, os, dos, dxs, nslots, ring_len;
  int silu;
};

// The sequence of token t: the last s with cu[s] <= t (uniform).
__device__ __forceinline__ int64_t find_seq(const int32_t *cu, int64_t nseq, int64_t t) {
  return wave_search(nseq, [&](int64_t s) { return cu[s] <= t; });
}
__device__ __forceinline__ auto edges_of(const int32_t *cu) {
  return [=](int64_t s) { return static_cast<int64_t>(cu[s]); };
}

// Where a sequence's ring is, and how many tokens went before.
struct RingOf {
  int64_t slot;
  int seen;
};
__device__ __forceinline__ RingOf ring_of(const ConvVarParams &p, int64_t s) {
  if (!p.ring) return {-1, 0};
  return {p.slots ? p.slots[s] : s, p.seen ? p.seen[s] : 0};
}
// The input `back` tokens before a sequence's first one, from its ring.
template <int IO, int NV>
__device__ __forceinline__ void ring_input(const ConvVarParams &p, const RingOf &ring, int back, int64_t c0, float (&v)[NV]) {
  const int pos = ring.seen - back;
  const bool there = pos >= 0 && ring.slot >= 0 && ring.slot < p.nslots;
  const int64_t at = there ? (ring.slot * p.channels + c0) * p.ring_len + static_cast<uint32_t>(pos) % static_cast<uint32_t>(p.ring_len) : 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) v[k] = there ? load_io<IO>(p.ring, at + k * p.ring_len) : 0.0f;
}

// The weights of the workgroup's 64 NV channels, through LDS: a lane's own NV
// rows are 16 NV bytes apart from the next lane's, and read from memory they
// cost a wave more of the L1's time than a run's inputs and outputs.  The row
// of channel c is kept at place_of(c), which spreads the lanes' reads over the
// banks.
template <int NV>
struct Weights {
  float4 w[NV > 1 ? 64 * NV : 1];
  static __device__ __forceinline__ int place_of(int c) { return c ^ ((c / NV) & (NV - 1)); }
  static __device__ __forceinline__ float4 row(const ConvVarParams &p, int64_t c) {
    const Row4 r = reinterpret_cast<const Row4 *>(p.w)[c];
    return make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
  }
  // (a barrier belongs between the two)
  __device__ __forceinline__ void fill(const ConvVarParams &p, int64_t first) {
    if constexpr (NV > 1) {
#pragma unroll
      for (int i = 0; i < NV / kRows; ++i) {
        const int c = i * 64 * kRows + threadIdx.x;
        if (first + c < p.channels) w[place_of(c)] = row(p, first + c);
      }
    }
  }
  __device__ __forceinline__ void take(const ConvVarParams &p, int64_t c0, int lane, float (&wr)[kW][NV], float (&b)[NV]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const float4 v = NV > 1 ? w[place_of(lane * NV + k)] : row(p, c0 + k);
      wr[0][k] = v.x; wr[1][k] = v.y; wr[2][k] = v.z; wr[3][k] = v.w;
      b[k] = p.bias ? p.bias[c0 + k] : 0.0f;
    }
  }
};

// A sequence's last inputs into its ring.  The run with the sequence's first
// token does it, which alone reads what the ring held before (run_pieces).
template <int IO, int NV>
__device__ __forceinline__ void keep_inputs(const ConvVarParams &p, const RingOf &ring, int64_t first, int64_t end, int64_t c0) {
  const int64_t slot = ring.slot, seen = ring.seen > 0 ? ring.seen : 0;
  if (end <= first || slot < 0 || slot >= p.nslots) return;
#pragma unroll 1
  for (int64_t t = end - first > p.ring_len ? end - p.ring_len : first; t < end; t += 4) {   // four loads in flight
    Vec<IO, NV> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i < end) v[i].load(p.x, (t + i) * p.xs + c0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i < end) {
        const int64_t at = (slot * p.channels + c0) * p.ring_len +
                           static_cast<uint64_t>(seen + t + i - first) % static_cast<uint32_t>(p.ring_len);
#pragma unroll
        for (int k = 0; k < NV; ++k) store_one<IO>(p.ring, at + k * p.ring_len, v[i].get(k));
      }
  }
}

template <int IO, int NV, int RUN>
__global__ void __launch_bounds__(64 * kRows, 4) conv_var_fwd_kernel(const ConvVarParams p) {
  const int lane = threadIdx.x & 63;
  const int row = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRows + row) * RUN;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * 64 + lane) * NV;
  __shared__ Weights<NV> weights;
  weights.fill(p, c0 - lane * NV);
  const int64_t s = t0 < p.total ? find_seq(p.cu, p.nseq, t0) : 0;
  if constexpr (NV > 1) __syncthreads();
  if (t0 >= p.total || c0 >= p.channels) return;
  const int n = static_cast<int>(p.total - t0 < RUN ? p.total - t0 : RUN);

  Vec<IO, NV> in[RUN + kW - 1];
#pragma unroll
  for (int i = 0; i < RUN + kW - 1; ++i) {
    const int64_t t = t0 + i - (kW - 1);
    if (t >= 0 && i < n + kW - 1) in[i].load(p.x, t * p.xs + c0);
    else in[i].zero();
  }
  float w[kW][NV], bias[NV];
  weights.take(p, c0, lane, w, bias);
  RingOf ring = ring_of(p, s);   // (asked for with the two below, not behind them)
  const auto edge = edges_of(p.cu);
  if (n == RUN && inside_one(edge, s, t0, t0 + RUN)) {
    // the whole run and what it sees are inside one sequence: no branch
    // between the loads and their use (with the edge tests of every token in
    // between the compiler kept few loads in flight: 216 us where this took
    // 88 at 16384 x 5376 bf16; 85 now)
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      float acc[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        acc[k] = bias[k];
#pragma unroll
        for (int j = kW - 1; j >= 0; --j) acc[k] = fmaf(w[j][k], in[i + j].get(k), acc[k]);
        if (p.silu) acc[k] = silu_f(acc[k]);
      }
      put<IO, NV>(p.out, (t0 + i) * p.os + c0, acc);
    }
    return;
  }
  // A run with an edge in it, sequence by sequence: what lies before the
  // piece's first token once, then its tokens with the last inputs rolling.
  run_pieces(edge, p.nseq, p.total, t0, n, s, [&](int64_t of, int from, int to, int64_t place, int64_t end) {
    if (of != s) ring = ring_of(p, of);
    float win[kW - 1][NV];   // the last inputs, oldest first
#pragma unroll
    for (int back = 1; back < kW; ++back) {
      float (&h)[NV] = win[kW - 1 - back];
      if (place >= back) {
        Vec<IO, NV> v;
        v.load(p.x, (t0 + from - back) * p.xs + c0);
#pragma unroll
        for (int k = 0; k < NV; ++k) h[k] = v.get(k);
      } else {
        ring_input<IO, NV>(p, ring, back - static_cast<int>(place), c0, h);
      }
    }
    if (p.ring && place == 0) keep_inputs<IO, NV>(p, ring, t0 + from, end < p.total ? end : p.total, c0);
    // (the run's inputs once more, four tokens at a time: sharing the
    // registers above with this path doubled the kernel's)
#pragma unroll 1
    for (int i = from; i < to; i += 4) {
      Vec<IO, NV> now[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + q < to) now[q].load(p.x, (t0 + i + q) * p.xs + c0);
        else now[q].zero();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (i + q >= to) break;
        float acc[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const float v = now[q].get(k);
          acc[k] = fmaf(w[kW - 1][k], v, bias[k]);
#pragma unroll
          for (int j = kW - 2; j >= 0; --j) acc[k] = fmaf(w[j][k], win[j][k], acc[k]);
          if (p.silu) acc[k] = silu_f(acc[k]);
#pragma unroll
          for (int j = 0; j < kW - 2; ++j) win[j][k] = win[j + 1][k];
          win[kW - 2][k] = v;
        }
        put<IO, NV>(p.out, (t0 + i + q) * p.os + c0, acc);
      }
    }
  });
}

// Backward.  At token t the pre-activation is formed again from x, and
// da_t = dout_t act'(pre_t) goes to the gradients of the inputs it saw: the
// run's pending dx of tokens t-3..t are in registers, and token t-3's is
// complete.  The three tokens after the run are walked for what they give to
// the run's last ones; their weight gradients belong to the next run.  The
// weight and bias gradients of the workgroup's four runs meet in LDS and go
// out as one row of partial sums.
template <int IO, int NV, int RUN>
__global__ void __launch_bounds__(64 * kRows) conv_var_bwd_kernel(const ConvVarParams p) {
  __shared__ float sum[kRows - 1][kW + 1][NV][64];
  const int lane = threadIdx.x & 63;
  const int row = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRows + row) * RUN;
  const int64_t c0 = (static_cast<int64_t>(blockIdx.y) * 64 + lane) * NV;
  const bool live = c0 < p.channels;
  __shared__ Weights<NV> weights;
  weights.fill(p, c0 - lane * NV);
  const int64_t of_first = t0 < p.total ? find_seq(p.cu, p.nseq, t0) : 0;
  if constexpr (NV > 1) __syncthreads();
  float dw[kW + 1][NV];
#pragma unroll
  for (int j = 0; j <= kW; ++j)
#pragma unroll
    for (int k = 0; k < NV; ++k) dw[j][k] = 0.0f;

  if (live && t0 < p.total) {
    const int64_t stop = t0 + RUN < p.total ? t0 + RUN : p.total;              // end of the run
    const int64_t walk = stop + kW - 1 < p.total ? stop + kW - 1 : p.total;            // and of the walk
    float w[kW][NV], bias[NV];
    weights.take(p, c0, lane, w, bias);
    int64_t s = of_first;
    const auto edge = edges_of(p.cu);
    int64_t end = edge(s + 1);
    int64_t pos = t0 - first_token(edge, s);
    if (walk - t0 == RUN + kW - 1 && inside_one(edge, s, t0, walk)) {
      // the run and all that it sees are inside one sequence.  Token i's input
      // and pending gradient are in place i % 4, so nothing moves along and
      // nothing is tested (16384 x 5376 bf16: 126 us where the general walk
      // takes 131).  Single channels ask for the next four tokens before they
      // compute four (16384 x 1003: 40 us for 58); several channels would need
      // 144 registers for that, which leaves three waves a SIMD (144 us).
      static_assert(kW == 4 && RUN % 8 == 0, "places, and blocks in pairs");
      float in[4][NV], pend[4][NV];
      Vec<IO, NV> x0[4], g0[4], x1[4], g1[4];
      auto ask = [&](Vec<IO, NV> (&xv)[4], Vec<IO, NV> (&gv)[4], int i0) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < 3 || i0 < RUN) {
            xv[q].load(p.x, (t0 + i0 + q) * p.xs + c0);
            gv[q].load(p.dout, (t0 + i0 + q) * p.dos + c0);
          }
      };
      // token i0 + q, which completes token i0 + q - 3
      auto token = [&](const Vec<IO, NV> &x, const Vec<IO, NV> &g, int i0, auto place, auto own) {
        constexpr int Q = decltype(place)::value;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          in[Q][k] = x.get(k);
          float pre = bias[k];
#pragma unroll
          for (int back = 0; back < kW; ++back) pre = fmaf(w[kW - 1 - back][k], in[(Q - back) & 3][k], pre);
          float da = g.get(k);
          if (p.silu) {
            const float sg = fast_rcp(1.0f + fast_exp2(-pre * kLog2e));
            da *= fmaf(pre * sg, 1.0f - sg, sg);
          }
          pend[Q][k] = w[kW - 1][k] * da;
#pragma unroll
          for (int back = 1; back < kW; ++back) pend[(Q - back) & 3][k] = fmaf(w[kW - 1 - back][k], da, pend[(Q - back) & 3][k]);
          if constexpr (decltype(own)::value) {
#pragma unroll
            for (int back = 0; back < kW; ++back) dw[kW - 1 - back][k] = fmaf(da, in[(Q - back) & 3][k], dw[kW - 1 - back][k]);
            dw[kW][k] += da;
          }
        }
        if (Q == 3 || i0 > 0) put<IO, NV>(p.dx, (t0 + i0 + Q - 3) * p.dxs + c0, pend[(Q + 1) & 3]);
      };
      auto block = [&](const Vec<IO, NV> (&xv)[4], const Vec<IO, NV> (&gv)[4], int i0, auto own) {
        static_for(std::make_integer_sequence<int, decltype(own)::value ? 4 : 3>{},
                   [&](auto q) { token(xv[decltype(q)::value], gv[decltype(q)::value], i0, q, own); });
      };
#pragma unroll
      for (int j = 0; j < kW - 1; ++j) {
        x1[j].load(p.x, (t0 - (kW - 1) + j) * p.xs + c0);
      }
      if constexpr (NV == 1) ask(x0, g0, 0);
#pragma unroll
      for (int j = 0; j < kW - 1; ++j)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          in[j + 1][k] = x1[j].get(k);
          pend[j + 1][k] = 0.0f;   // of tokens before the run, which others complete
        }
      if constexpr (NV == 1) {
#pragma unroll 1
        for (int i = 0; i < RUN; i += 8) {
          ask(x1, g1, i + 4);
          block(x0, g0, i, std::true_type{});
          ask(x0, g0, i + 8);
          block(x1, g1, i + 4, std::true_type{});
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < RUN; i += 4) {
          ask(x0, g0, i);
          block(x0, g0, i, std::true_type{});
        }
        ask(x0, g0, RUN);
      }
      block(x0, g0, RUN, std::false_type{});
    } else {
      // the last three inputs, oldest first, and the pending gradients
      float win[kW][NV], pend[kW][NV];
#pragma unroll
      for (int j = 0; j < kW - 1; ++j) {
        const int64_t t = t0 - (kW - 1) + j;
        Vec<IO, NV> v;
        if (t >= 0) v.load(p.x, t * p.xs + c0);
        else v.zero();
#pragma unroll
        for (int k = 0; k < NV; ++k) win[j][k] = v.get(k);
      }
#pragma unroll
      for (int j = 0; j < kW; ++j)
#pragma unroll
        for (int k = 0; k < NV; ++k) pend[j][k] = 0.0f;
      constexpr int STEP = NV == 1 ? 4 * kStep : kStep;   // single channels: as many bytes in flight
      for (int64_t tb = t0; tb < walk + kW - 1; tb += STEP) {
        Vec<IO, NV> xv[STEP], gv[STEP];
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          if (tb + i < walk) {
            xv[i].load(p.x, (tb + i) * p.xs + c0);
            gv[i].load(p.dout, (tb + i) * p.dos + c0);
          } else {
            xv[i].zero();
            gv[i].zero();
          }
        }
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          const int64_t t = tb + i;
          if (t < walk) {
            while (t >= end && s + 1 < p.nseq) {
              ++s;
              end = edge(s + 1);
              pos = t - first_token(edge, s);
            }
            float da[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
              win[kW - 1][k] = xv[i].get(k);
              da[k] = fmaf(w[kW - 1][k], win[kW - 1][k], bias[k]);
            }
#pragma unroll
            for (int back = 1; back < kW; ++back)
              if (pos >= back) {
#pragma unroll
                for (int k = 0; k < NV; ++k) da[k] = fmaf(w[kW - 1 - back][k], win[kW - 1 - back][k], da[k]);
              }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
              const float pre = da[k];
              float d = gv[i].get(k);
              if (p.silu) {
                const float sg = fast_rcp(1.0f + fast_exp2(-pre * kLog2e));
                d *= fmaf(pre * sg, 1.0f - sg, sg);
              }
              da[k] = d;
            }
            const bool mine = t < stop;
#pragma unroll
            for (int back = 0; back < kW; ++back)
              if (pos >= back) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                  pend[kW - 1 - back][k] = fmaf(w[kW - 1 - back][k], da[k], pend[kW - 1 - back][k]);
                  if (mine) dw[kW - 1 - back][k] = fmaf(da[k], win[kW - 1 - back][k], dw[kW - 1 - back][k]);
                }
              }
            if (mine) {
#pragma unroll
              for (int k = 0; k < NV; ++k) dw[kW][k] += da[k];
            }
            ++pos;
          }
          const int64_t done = t - (kW - 1);   // its gradient is complete
          if (done >= t0 && done < stop) put<IO, NV>(p.dx, done * p.dxs + c0, pend[0]);
#pragma unroll
          for (int j = 0; j < kW - 1; ++j)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
              pend[j][k] = pend[j + 1][k];
              win[j][k] = win[j + 1][k];
            }
#pragma unroll
          for (int k = 0; k < NV; ++k) pend[kW - 1][k] = 0.0f;
        }
      }
    }
  }
  if (row > 0) {
#pragma unroll
    for (int j = 0; j <= kW; ++j)
#pragma unroll
      for (int k = 0; k < NV; ++k) sum[row - 1][j][k][lane] = dw[j][k];
  }
  __syncthreads();
  if (row == 0 && live) {
#pragma unroll
    for (int j = 0; j <= kW; ++j)
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float v = dw[j][k];
#pragma unroll
        for (int q = 0; q < kRows - 1; ++q) v += sum[q][j][k][lane];
        p.part[(static_cast<int64_t>(blockIdx.x) * (kW + 1) + j) * p.channels + c0 + k] = v;
      }
  }
}

// Sum of the partial rows, four threads a column, each its quarter in order;
// in 64 bits, so that the sum over many tokens keeps 32.
__global__ void __launch_bounds__(256) conv_var_reduce_kernel(const float *part, float *dweight, float *dbias,
                                                              int64_t rows, int64_t channels) {
  __shared__ double sum[4][64];
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane, cols = (kW + 1) * channels;
  double v = 0.0;
  if (col < cols) {
    const int64_t to = rows * (q + 1) / 4;
    int64_t r = rows * q / 4;
    for (; r + 8 <= to; r += 8) {   // eight loads in flight
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = part[(r + i) * cols + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += f[i];
    }
    for (; r < to; ++r) v += part[r * cols + col];
  }
  sum[q][lane] = v;
  __syncthreads();
  if (q == 0 && col < cols) {
    const float total = static_cast<float>((sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]));
    const int64_t j = col / channels, c = col - j * channels;
    if (j < kW) dweight[c * kW + j] = total;
    else if (dbias) dbias[c] = total;
  }
}

ConvVarParams conv_params(const causal_conv1d_varlen_args_t *a) {
  ConvVarParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.w = a->weight; p.bias = a->bias; p.cu = a->cu_seqlens;
  p.total = a->total; p.nseq = a->nseq; p.channels = a->channels;
  p.silu = a->act == SSM_ACT_SILU;
  return p;
}

// Waves of a launch whose runs are `run` tokens long.
int64_t run_waves(const causal_conv1d_varlen_args_t *a, int nv, int run) {
  return (a->total + run - 1) / run * ((a->channels + 64 * nv - 1) / (64 * nv));
}
// A launch of few waves lasts as long as one of its runs with an edge, so runs
// are short below eight long ones a compute unit.  Measured short / long (us),
// forward, 16 sequences from and to their rings: 500 x 1024 9.5 / 13.0, 3500 x
// 2304 16.9 / 18.9, and above the limit 8192 x 2304 37 / 27, 16384 x 5376 108 /
// 76; backward: 500 x 1024 13.4 / 26.7, 3500 x 2304 24 / 33, and above it 8192 x
// 2304 45 / 39, 16384 x 5376 160 / 123.
constexpr int kFewWaves = 8;
int fwd_run(const causal_conv1d_varlen_args_t *a, int nv) {
  return run_waves(a, nv, kFwdRun) < kFewWaves * static_cast<int64_t>(cu_count_cached()) ? kShortRun : kFwdRun;
}
int bwd_run(const causal_conv1d_varlen_args_t *a, int nv) {
  return run_waves(a, nv, kBwdRun) < kFewWaves * static_cast<int64_t>(cu_count_cached()) ? kShortBwdRun : kBwdRun;
}
int64_t blocks_of(int64_t total, int run) { return (total + kRows * run - 1) / (kRows * run); }

// 16-byte accesses need whole and aligned rows of them
bool wide_rows(int32_t io, int64_t channels, const void *p, int64_t stride) {
  const int nv = io == SSM_F32 ? 4 : 8;
  return channels % nv == 0 && aligned16(p) && stride % nv == 0;
}

// launch(io, channels of a lane): VEC of 16 bits, 4 of 32, or single ones.
template <int VEC, typename F>
void by_type(int32_t io, bool wide, std::integral_constant<int, VEC>, F &&launch) {
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, VEC> vec;
  const integral_constant<int, SSM_BF16> bf16;
  const integral_constant<int, SSM_F16> f16;
  const integral_constant<int, SSM_F32> f32;
  if (io == SSM_BF16) wide ? launch(bf16, vec) : launch(bf16, one);
  else if (io == SSM_F16) wide ? launch(f16, vec) : launch(f16, one);
  else wide ? launch(f32, integral_constant<int, 4>{}) : launch(f32, one);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int causal_conv1d_varlen_fwd(const causal_conv1d_varlen_args_t *a, void *stream_ptr) {
  const int st = causal_conv1d_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  ConvVarParams p = conv_params(a);
  p.out = a->out; p.os = a->out_stride;
  p.ring = a->conv_state; p.nslots = a->state_slots; p.ring_len = a->state_len;
  p.seen = a->cache_seqlens; p.slots = a->slots;
  const bool wide = wide_rows(a->io_dtype, a->channels, a->x, a->x_stride) &&
                    wide_rows(a->io_dtype, a->channels, a->out, a->out_stride);
  const int nv = !wide ? 1 : a->io_dtype == SSM_F32 ? 4 : 8;
  const int run = fwd_run(a, nv);
  const int64_t gx = blocks_of(a->total, run), gy = (a->channels + 64 * nv - 1) / (64 * nv);
  if (gy > 65535 || !grid_fits(gx, 64 * kRows)) return SSM_ERR_SHAPE;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), block(64 * kRows);
  auto launch = [&](auto io, auto vec) {
    constexpr int IO = decltype(io)::value, NV = decltype(vec)::value;
    const auto fn = run == kFwdRun ? conv_var_fwd_kernel<IO, NV, kFwdRun> : conv_var_fwd_kernel<IO, NV, kShortRun>;
    hipLaunchKernelGGL(fn, grid, block, 0, stream, p);
  };
  by_type(a->io_dtype, wide, std::integral_constant<int, 8>{}, launch);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

extern "C" int causal_conv1d_varlen_bwd_workspace_size(const causal_conv1d_varlen_args_t *a, size_t *bytes) {
  const int st = causal_conv1d_varlen_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  // the shorter runs' partial sums, whichever the call's strides let it take
  *bytes = static_cast<size_t>(blocks_of(a->total, bwd_run(a, kBwdVec))) * (kW + 1) * a->channels * sizeof(float);
  return SSM_OK;
}

extern "C" int causal_conv1d_varlen_bwd(const causal_conv1d_varlen_args_t *a, void *stream_ptr) {
  size_t need = 0;
  const int st = causal_conv1d_varlen_bwd_workspace_size(a, &need);
  if (st != SSM_OK) return st;
  if (!a->workspace || a->workspace_bytes < need) return SSM_ERR_WORKSPACE;
  ConvVarParams p = conv_params(a);
  p.dout = a->dout; p.dos = a->dout_stride;
  p.dx = a->dx; p.dxs = a->dx_stride;
  p.part = static_cast<float *>(a->workspace);
  const bool wide = wide_rows(a->io_dtype, a->channels, a->x, a->x_stride) &&
                    wide_rows(a->io_dtype, a->channels, a->dout, a->dout_stride) &&
                    wide_rows(a->io_dtype, a->channels, a->dx, a->dx_stride);
  const int nv = !wide ? 1 : a->io_dtype == SSM_F32 ? 4 : kBwdVec;
  const int run = bwd_run(a, nv);
  const int64_t gx = blocks_of(a->total, run), gy = (a->channels + 64 * nv - 1) / (64 * nv);
  if (gy > 65535 || !grid_fits(gx, 64 * kRows)) return SSM_ERR_SHAPE;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), block(64 * kRows);
  auto launch = [&](auto io, auto vec) {
    constexpr int IO = decltype(io)::value, NV = decltype(vec)::value;
    const auto fn = run == kBwdRun ? conv_var_bwd_kernel<IO, NV, kBwdRun> : conv_var_bwd_kernel<IO, NV, kShortBwdRun>;
    hipLaunchKernelGGL(fn, grid, block, 0, stream, p);
  };
  by_type(a->io_dtype, wide, std::integral_constant<int, kBwdVec>{}, launch);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e);
  const int64_t cols = (kW + 1) * a->channels;
  hipLaunchKernelGGL(conv_var_reduce_kernel, dim3(static_cast<unsigned>((cols + 63) / 64)), dim3(256), 0, stream, p.part,
                     a->dweight, a->dbias, gx, a->channels);
  e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}
