// ssd_varlen.hip -- the Mamba-2 chunked scan over packed tokens
// (ssd_varlen_fwd): prompts of several lengths from and to a cache of states,
// and the training forward, which keeps every chunk's entering state in 8
// bits.
//
// The evaluation is ssd.hip's: per chunk of Q = 64 tokens with dt' the step,
// cs its running sum times A, S the (headdim x dstate) state entering it,
//   M[t][tau] = (C_t . B_tau) exp(cs_t - cs_tau) dt'_tau      (tau <= t)
//   Y         = M X + diag(exp(cs)) C S^T
//   S        <- exp(cs_end) S + X^T diag(exp(cs_end - cs) dt') B
// with M and S entering their products as a bf16 head and tail.  The weighted
// X of the state update enters in three parts (all 24 bits) and the running
// sum is kept in two floats: the state is a 32-bit output, and its 8-bit form
// is decided by it.
//
// What bounds it is the chain of a chunk's dependent steps, not HBM: the chunks
// of a (sequence, head) follow each other.  So:
// - a workgroup of eight waves runs two heads of a group, which share B and C;
// - the next chunk's x, B and C go from global memory straight into the other
//   half of a double buffer in LDS while this chunk is computed (no registers,
//   and the latency, about a third of a chunk's time before, is hidden), and
//   its steps are summed at this chunk's end;
// - tiles stay as they lie in memory, token by token, and are read across by
//   the transposing LDS load, so nothing is rearranged on the way;
// - two barriers a chunk: data there, M there.
// With few (sequence, head) pairs the sequence is cut into segments; a first
// launch finds their end states from zero (packed_scan_kernel<N, false>), and
// the second starts every segment from the states carried over.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_util.h"
#include "packed_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kPair = 2;   // heads of a workgroup

struct ScanParams {
  const uint16_t *x, *dt, *B, *C, *z;
  const float *A, *D, *dt_bias;
  uint16_t *out;
  float *ws_state, *ws_decay;   // segments: end states (and the cached states' copies), decays
  const int32_t *cu, *seen, *slots;
  float *cache;
  int8_t *codes;
  float *scales;
  int64_t xs, dts, bs, cs, zs, os;
  int64_t total, max_seqlen, cache_slots, nheads, ngroups, pairs, seg_chunks;
  int D_per_channel, nseg;
  StepRule step;
};

template <int N, bool FULL>
struct ScanLds {
  uint16_t B[2][kQ * N];                       // [t][n]
  uint16_t x[2][kPair][kQ * kP];               // [t][p]
  uint16_t C[FULL ? 2 : 1][FULL ? kQ * N : 8];       // [t][n]
  uint16_t M[FULL ? kPair : 1][2][FULL ? kQ * kQ : 8];   // [t][tau] head, tail
  // running sum, step, exp(cs), and the state update's weight, per token
  float cs[2][kPair][kQ], dt[2][kPair][kQ], e[2][kPair][kQ], w[2][kPair][kQ];
};

// 16-byte pieces of a row-major tile of `rows` tokens straight into LDS, the
// pieces of wave w.  A wave writes one KiB in order, so the tile's permutation
// (tile_at, its own inverse) is applied to where each lane reads.  Tokens at
// and after `len` repeat the last one: their steps are 0, and what they give
// reaches no output.
template <int ROW_LEN>
__device__ __forceinline__ void tile_to_lds(uint16_t *tile, const uint16_t *from, int64_t stride, int len, int w, int nw,
                                            int lane) {
  constexpr int G = ROW_LEN / 8;
  for (int i = w; i < kQ * G / 64; i += nw) {
    const int piece = i * 64 + lane, row = piece / G, t = row < len ? row : len - 1;
    const uint16_t *src = from + t * stride + (tile_at<ROW_LEN>(row, (piece % G) * 8) - row * ROW_LEN);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)(tile + i * 512), 16, 0, 0);
  }
}

// A barrier for LDS alone: what is on its way from global memory stays so.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int N, bool FULL>
__global__ void __launch_bounds__(512, FULL ? 2 : 4) packed_scan_kernel(const ScanParams p) {
  constexpr int KN = N / 32;   // K steps over dstate
  constexpr int NT = N / 16;   // state tiles along dstate
  extern __shared__ __attribute__((aligned(16))) char smem[];
  ScanLds<N, FULL> &sm = *reinterpret_cast<ScanLds<N, FULL> *>(smem);
  const int tid = threadIdx.x, l = tid & 63, r = l & 15, kq = l >> 4;
  const int w8 = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hw = w8 >> 2, w = w8 & 3;   // which head of the pair; its channels 16w..16w+15
  // the pair: heads h0 and h0 + 1 of group g
  const int64_t s = blockIdx.x / p.pairs, pr = blockIdx.x - s * p.pairs;
  const int64_t hpg = p.nheads / p.ngroups, per = (hpg + kPair - 1) / kPair;
  const int64_t g = pr / per, in_group = (pr - g * per) * kPair + hw;
  const bool alive = in_group < hpg;   // an odd group's last pair: the second head runs along and writes nothing
  const int64_t h = g * hpg + (alive ? in_group : in_group - 1);
  const int64_t SH = static_cast<int64_t>(gridDim.x) / p.pairs * p.nheads, sh = s * p.nheads + h;
  const Seq q = sequence(p.cu, p.total, p.max_seqlen, s);
  // the full pass dispatches its last segments first: those of the longest sequences
  const int64_t seg = FULL ? static_cast<int64_t>(gridDim.y) - 1 - blockIdx.y : blockIdx.y;
  const int64_t c_begin = seg * p.seg_chunks;
  const int64_t c_end = c_begin + p.seg_chunks < q.chunks ? c_begin + p.seg_chunks : q.chunks;
  const bool last_seg = c_end >= q.chunks;
  if (seg > 0 && c_begin >= q.chunks) return;
  if (!FULL && last_seg) return;   // the first launch runs the segments that have one after them
  int64_t slot = p.slots ? p.slots[s] : s;
  if (slot >= p.cache_slots) slot = -1;
  const bool cached = p.cache && slot >= 0 && p.seen && p.seen[s] > 0;

  const uint16_t *xb = p.x + q.first * p.xs + h * kP;
  const uint16_t *zb = p.z ? p.z + q.first * p.zs + h * kP : nullptr;
  const uint16_t *Bb = p.B + q.first * p.bs + g * N, *Cb = p.C + q.first * p.cs + g * N;
  const uint16_t *dtb = p.dt + q.first * p.dts + h;
  uint16_t *ob = p.out + q.first * p.os + h * kP;
  const float Ah = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
  float *state_ws = p.ws_state + sh * kP * N;   // segment k's at k * SH * kP * N
  const int srow = (16 * w + r) * N + 4 * kq;   // this lane's first state element in a (p, n) block

  auto chunk_len = [&](int64_t c) { return static_cast<int>(q.len - c * kQ < kQ ? q.len - c * kQ : kQ); };
  auto fetch = [&](int64_t c, int b) {
    const int64_t t0 = c * kQ;
    const int len = chunk_len(c);
    tile_to_lds<kP>(sm.x[b][hw], xb + t0 * p.xs, p.xs, len, w, 4, l);
    tile_to_lds<N>(sm.B[b], Bb + t0 * p.bs, p.bs, len, w8, 8, l);
    if constexpr (FULL) tile_to_lds<N>(sm.C[b], Cb + t0 * p.cs, p.cs, len, w8, 8, l);
  };
  // a chunk's raw steps, and what the chunk needs of them (wave 0 of each head)
  auto raw_steps = [&](int64_t c) { return l < chunk_len(c) ? bf2f(dtb[(c * kQ + l) * p.dts]) : 0.0f; };
  auto put_steps = [&](int64_t c, int b, float raw) {
    float v;
    const float d = chunk_step(p.step, raw, bias, l < chunk_len(c), v);
    const TwoSum cs = running_sum(d, Ah);
    const float eh = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cs.hi), 63));
    const float el = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cs.lo), 63));
    sm.cs[b][hw][l] = cs.hi;
    sm.dt[b][hw][l] = d;
    sm.e[b][hw][l] = exp_diff(cs.hi, cs.lo, 0.0f, 0.0f);
    sm.w[b][hw][l] = exp_diff(eh, el, cs.hi, cs.lo) * d;
  };

  // ---- state, transposed: wave w holds S[p = 16w + r][n = 16 nt + 4kq + i].
  // The state pass starts segment 0 from the cached state and the others from
  // zero; the full pass starts segment k from E_{k-1} + P_{k-1} (E_{k-2} + ...).
  // The last segment's workgroup writes the cache while others may still be
  // starting, so a sequence of several segments reads it in the state pass
  // alone: segment 0's start is a copy that the state pass leaves behind the
  // E's.
  f32x4 accs[NT];
  {
    const float *start = nullptr;
    if (cached && seg == 0)
      start = (!FULL || last_seg) ? p.cache + (slot * p.nheads + h) * kP * N : state_ws + (p.nseg - 1) * SH * kP * N;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 v = start ? *reinterpret_cast<const float4 *>(start + srow + 16 * nt) : make_float4(0, 0, 0, 0);
      accs[nt] = (f32x4){v.x, v.y, v.z, v.w};
      if (!FULL && start && alive)
        *reinterpret_cast<float4 *>(state_ws + (p.nseg - 1) * SH * kP * N + srow + 16 * nt) = v;
    }
  }
  if (FULL) {
    for (int64_t j = 0; j < seg; ++j) {
      const float P = p.ws_decay[j * SH + sh];
      const float *E = state_ws + j * SH * kP * N + srow;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 e = *reinterpret_cast<const float4 *>(E + 16 * nt);
        accs[nt] = (f32x4){fmaf(P, accs[nt][0], e.x), fmaf(P, accs[nt][1], e.y), fmaf(P, accs[nt][2], e.z),
                           fmaf(P, accs[nt][3], e.w)};
      }
    }
  }
  if constexpr (FULL) {   // M's blocks above the diagonal stay zero
    for (int i = tid; i < kPair * 2 * kQ * kQ / 8; i += 512) reinterpret_cast<uint4 *>(&sm.M[0][0][0])[i] = make_uint4(0, 0, 0, 0);
  }
  float Dv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int pc = 16 * w + 4 * kq;   // this lane's channels of Y
  if (FULL && p.D) {
#pragma unroll
    for (int i = 0; i < 4; ++i) Dv[i] = p.D_per_channel ? p.D[h * kP + pc + i] : p.D[h];
  }
  float seg_decay = 1.0f;

  if (c_begin < c_end) {
    fetch(c_begin, 0);
    if (w == 0) put_steps(c_begin, 0, raw_steps(c_begin));
  }
  for (int64_t c = c_begin; c < c_end; ++c) {
    const int b = static_cast<int>((c - c_begin) & 1);
    const int64_t t0 = c * kQ;
    const int len = chunk_len(c);
    // this wave's part of the chunk's tiles is there; after the barrier every
    // wave's, and the last chunk's readers are done
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float raw = 0.0f;
    const bool more = c + 1 < c_end;
    if (w == 0 && more) raw = raw_steps(c + 1);
    uint2 zv[4] = {};
    if (FULL && zb) {
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
        if (16 * tb + r < len) zv[tb] = *reinterpret_cast<const uint2 *>(zb + (t0 + 16 * tb + r) * p.zs + pc);
    }
    if (more) fetch(c + 1, b ^ 1);
    const float *cs = sm.cs[b][hw], *dt = sm.dt[b][hw], *e0 = sm.e[b][hw], *we = sm.w[b][hw];
    uint16_t *X = sm.x[b][hw], *B = sm.B[b], *C = sm.C[FULL ? b : 0];

    if constexpr (FULL) {
      if (p.codes) {
        // the chunk's entering state in 8 bits: this lane holds 4 NT states of
        // row 16w + r, the row's others are 16, 32 and 48 lanes away
        uint32_t top = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = __float_as_uint(accs[nt][i]) & 0x7fffffffu;
            top = v > top ? v : top;
          }
        uint32_t o = __shfl_xor(top, 16);
        top = o > top ? o : top;
        o = __shfl_xor(top, 32);
        top = o > top ? o : top;
        float inv;
        const float scale = row_scale(top, inv);
        const int64_t row = ((q.entry + c) * p.nheads + h) * kP + 16 * w + r;
        if (alive) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t word = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              word |= (static_cast<uint32_t>(static_cast<int>(rintf(accs[nt][i] * inv))) & 0xffu) << (8 * i);
            *reinterpret_cast<uint32_t *>(p.codes + row * N + 16 * nt + 4 * kq) = word;
          }
          if (kq == 0) p.scales[row] = scale;
        }
      }

      // ---- M, from G^T = B C^T: lane holds (t = 16 wt + r, tau = 16 tb + 4kq + i),
      // tau <= t.  The second head's waves take the token blocks in the other
      // order, so that the two waves of a SIMD share the triangle's work.
      const int wt = hw ? 3 - w : w, t = 16 * wt + r;
      const float cst = cs[t];
      bf16x8 cop[KN];
#pragma unroll
      for (int kk = 0; kk < KN; ++kk) cop[kk] = frag<N>(l, C, 16 * wt, 32 * kk);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        if (tb > wt) break;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kk = 0; kk < KN; ++kk) acc = mfma(frag<N>(l, B, 16 * tb, 32 * kk), cop[kk], acc);
        const float4 cs4 = *reinterpret_cast<const float4 *>(&cs[16 * tb + 4 * kq]);
        const float4 dt4 = *reinterpret_cast<const float4 *>(&dt[16 * tb + 4 * kq]);
        const float csv[4] = {cs4.x, cs4.y, cs4.z, cs4.w}, dtv[4] = {dt4.x, dt4.y, dt4.z, dt4.w};
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = acc[i] * fast_exp2((cst - csv[i]) * kLog2e) * dtv[i];
          m[i] = 16 * tb + 4 * kq + i <= t ? v : 0.0f;
        }
        uint2 hi, lo;
        split_bf2(m[0], m[1], hi.x, lo.x);
        split_bf2(m[2], m[3], hi.y, lo.y);
        const int o = tile_at<kQ>(t, 16 * tb + 4 * kq);
        *reinterpret_cast<uint2 *>(&sm.M[hw][0][o]) = hi;
        *reinterpret_cast<uint2 *>(&sm.M[hw][1][o]) = lo;
      }
      lds_barrier();
    }

    // X across: lane (channel 16w + r, tokens 32kk + 8kq + i)
    bf16x8 xt[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) xt[kk] = frag_t<kP>(l, X, 32 * kk, 16 * w);

    if constexpr (FULL) {
      // ---- Y^T = S C^T diag(exp(cs)) + X^T M^T for this wave's channels and
      // every token: lane holds Y[t = 16 tb + r][p = 16w + 4kq + i].  The state
      // operand is this lane's own accumulators: the k index runs over the
      // states 32kk + 16a + 4kq + j (a < 2, j < 4) in that order for both
      // operands, and C's are the matching 8-byte pieces of its rows.
      f32x4 acc[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) acc[tb] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < KN; ++kk) {
        uint32_t sh_[4], sl_[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          split_bf2(accs[2 * kk + i / 4][i % 4], accs[2 * kk + i / 4][i % 4 + 1], sh_[i / 2], sl_[i / 2]);
        const bf16x8 shi = __builtin_bit_cast(bf16x8, make_uint4(sh_[0], sh_[1], sh_[2], sh_[3]));
        const bf16x8 slo = __builtin_bit_cast(bf16x8, make_uint4(sl_[0], sl_[1], sl_[2], sl_[3]));
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const uint2 c0 = *reinterpret_cast<const uint2 *>(&C[tile_at<N>(16 * tb + r, 32 * kk + 4 * kq)]);
          const uint2 c1 = *reinterpret_cast<const uint2 *>(&C[tile_at<N>(16 * tb + r, 32 * kk + 16 + 4 * kq)]);
          const bf16x8 cf = __builtin_bit_cast(bf16x8, make_uint4(c0.x, c0.y, c1.x, c1.y));
          acc[tb] = mfma(shi, cf, acc[tb]);
          acc[tb] = mfma(slo, cf, acc[tb]);
        }
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) acc[tb] *= e0[16 * tb + r];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
          if (32 * kk < 16 * (tb + 1)) {   // tau blocks at or before the token block
            acc[tb] = mfma(xt[kk], frag<kQ>(l, sm.M[hw][0], 16 * tb, 32 * kk), acc[tb]);
            acc[tb] = mfma(xt[kk], frag<kQ>(l, sm.M[hw][1], 16 * tb, 32 * kk), acc[tb]);
          }
      // ---- out = (Y + D x) * silu(z), four channels of a token
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const int t = 16 * tb + r;
        float xv[4], y[4];
        four(&X[tile_at<kP>(t, pc)], xv);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = fmaf(Dv[i], xv[i], acc[tb][i]);
        if (!p.D) {   // an infinite x times no D is not a NaN
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = acc[tb][i];
        }
        if (zb) {
          const float zf[4] = {__uint_as_float(zv[tb].x << 16), __uint_as_float(zv[tb].x & 0xffff0000u),
                               __uint_as_float(zv[tb].y << 16), __uint_as_float(zv[tb].y & 0xffff0000u)};
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] *= silu_f(zf[i]);
        }
        if (t < len && alive)
          *reinterpret_cast<uint2 *>(ob + (t0 + t) * p.os + pc) = make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
      }
    }

    // ---- S^T <- exp(cs_end) S^T + B^T (X w), X w in three bf16 parts
    const float dec = e0[kQ - 1];
    if constexpr (!FULL) seg_decay *= dec;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) accs[nt] *= dec;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const uint4 xw = __builtin_bit_cast(uint4, xt[kk]);
      uint32_t x0[4], x1[4], x2[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float a = bf2f(raw_bits(xw, i)) * we[32 * kk + 8 * kq + i];
        const float d = bf2f(raw_bits(xw, i + 1)) * we[32 * kk + 8 * kq + i + 1];
        split_bf2(a, d, x0[i / 2], x1[i / 2]);
        x2[i / 2] = pack_bf2(a - __uint_as_float(x0[i / 2] << 16) - __uint_as_float(x1[i / 2] << 16),
                             d - __uint_as_float(x0[i / 2] & 0xffff0000u) - __uint_as_float(x1[i / 2] & 0xffff0000u));
      }
      const bf16x8 f0 = __builtin_bit_cast(bf16x8, make_uint4(x0[0], x0[1], x0[2], x0[3]));
      const bf16x8 f1 = __builtin_bit_cast(bf16x8, make_uint4(x1[0], x1[1], x1[2], x1[3]));
      const bf16x8 f2 = __builtin_bit_cast(bf16x8, make_uint4(x2[0], x2[1], x2[2], x2[3]));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bf16x8 bt = frag_t<N>(l, B, 32 * kk, 16 * nt);
        accs[nt] = mfma(bt, f0, accs[nt]);
        accs[nt] = mfma(bt, f1, accs[nt]);
        accs[nt] = mfma(bt, f2, accs[nt]);
      }
    }
    if (w == 0 && more) put_steps(c + 1, b ^ 1, raw);
  }

  if (!alive) return;
  float *end = nullptr;
  if constexpr (FULL) {
    if (p.cache && slot >= 0 && last_seg) end = p.cache + (slot * p.nheads + h) * kP * N + srow;
  } else {
    end = state_ws + seg * SH * kP * N + srow;
    if (w == 0 && l == 0) p.ws_decay[seg * SH + sh] = seg_decay;
  }
  if (end) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      *reinterpret_cast<float4 *>(end + 16 * nt) = make_float4(accs[nt][0], accs[nt][1], accs[nt][2], accs[nt][3]);
  }
}

using VarFn = void (*)(const ScanParams);

VarFn var_fn(int64_t dstate, bool full) {
  switch (dstate) {
    case 32: return full ? packed_scan_kernel<32, true> : packed_scan_kernel<32, false>;
    case 64: return full ? packed_scan_kernel<64, true> : packed_scan_kernel<64, false>;
    default: return full ? packed_scan_kernel<128, true> : packed_scan_kernel<128, false>;
  }
}

unsigned var_lds(int64_t dstate, bool full) {
  switch (dstate) {
    case 32: return full ? sizeof(ScanLds<32, true>) : sizeof(ScanLds<32, false>);
    case 64: return full ? sizeof(ScanLds<64, true>) : sizeof(ScanLds<64, false>);
    default: return full ? sizeof(ScanLds<128, true>) : sizeof(ScanLds<128, false>);
  }
}

hipError_t launch_var(int64_t dstate, bool full, dim3 grid, hipStream_t stream, const ScanParams &p) {
  const VarFn fn = var_fn(dstate, full);
  const unsigned lds = var_lds(dstate, full);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(lds));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, grid, dim3(512), lds, stream, p);
  return hipGetLastError();
}

struct VarPlan {
  int nseg;
  int64_t pairs, seg_chunks;
  size_t off_decay, ws_bytes;
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Segments of the longest sequence; a shorter one has fewer.  One workgroup
// fills a compute unit's LDS at dstate 128.  The segment count is the one that
// the model of host_util.h finds fastest, the state pass costing about a
// quarter of a chunk's time for every chunk but the last segment's.
VarPlan var_plan(const ssd_varlen_args_t *a, int cus) {
  VarPlan pl{};
  int64_t nchunks = (a->max_seqlen + kQ - 1) / kQ;
  if (nchunks < 1) nchunks = 1;
  const int64_t hpg = a->nheads / a->ngroups;
  pl.pairs = a->ngroups * ((hpg + kPair - 1) / kPair);
  const int64_t SH = a->nseq * a->nheads;
  int64_t G = 1;
  if (a->seq_segments >= 1) {
    G = a->seq_segments;
  } else {
    // sequences of the longest one's length that hold all tokens
    const int64_t rows = (a->total / kQ + a->nseq + nchunks - 1) / nchunks;
    const int64_t blocks = (rows < a->nseq ? rows : a->nseq) * pl.pairs;
    G = split_segments(blocks, nchunks, cus, 0.25, 64, 2);
  }
  if (G > nchunks) G = nchunks;
  if (G > 65535) G = 65535;
  pl.seg_chunks = (nchunks + G - 1) / G;
  pl.nseg = static_cast<int>((nchunks + pl.seg_chunks - 1) / pl.seg_chunks);
  if (pl.nseg > 1) {
    // the segments' end states, and behind them a copy of the cached states
    pl.off_decay = up256(static_cast<size_t>(pl.nseg) * SH * kP * a->dstate * sizeof(float));
    pl.ws_bytes = pl.off_decay + up256(static_cast<size_t>(pl.nseg - 1) * SH * sizeof(float));
  }
  return pl;
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int ssd_varlen_fwd_workspace_size(const ssd_varlen_args_t *a, size_t *bytes) {
  const int st = ssd_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = var_plan(a, cu_count_cached()).ws_bytes;
  return SSM_OK;
}

extern "C" int ssd_varlen_fwd(const ssd_varlen_args_t *a, void *stream_ptr) {
  const int st = ssd_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  const VarPlan pl = var_plan(a, cu_count_cached());
  if (pl.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < pl.ws_bytes)) return SSM_ERR_WORKSPACE;
  if (pl.ws_bytes > 0 && !aligned16(a->workspace)) return SSM_ERR_UNSUPPORTED;
  const int64_t blocks = a->nseq * pl.pairs;
  if (blocks > 0x7fffffffLL) return SSM_ERR_SHAPE;
  ScanParams p{};
  p.x = static_cast<const uint16_t *>(a->x); p.xs = a->x_stride;
  p.dt = static_cast<const uint16_t *>(a->dt); p.dts = a->dt_stride;
  p.B = static_cast<const uint16_t *>(a->B); p.bs = a->B_stride;
  p.C = static_cast<const uint16_t *>(a->C); p.cs = a->C_stride;
  p.z = static_cast<const uint16_t *>(a->z); p.zs = a->z_stride;
  p.out = static_cast<uint16_t *>(a->out); p.os = a->out_stride;
  p.A = a->A; p.D = a->D; p.dt_bias = a->dt_bias;
  p.D_per_channel = a->D_per_channel;
  p.step = {a->dt_softplus, a->dt_limit, a->dt_min, a->dt_max};
  p.nheads = a->nheads; p.ngroups = a->ngroups; p.pairs = pl.pairs;
  p.cu = a->cu_seqlens; p.total = a->total; p.max_seqlen = a->max_seqlen;
  p.cache = a->ssm_state; p.cache_slots = a->state_slots; p.seen = a->cache_seqlens; p.slots = a->slots;
  p.codes = a->checkpoints; p.scales = a->checkpoint_scales;
  p.nseg = pl.nseg; p.seg_chunks = pl.seg_chunks;
  if (pl.nseg > 1) {
    char *ws = static_cast<char *>(a->workspace);
    p.ws_state = reinterpret_cast<float *>(ws);
    p.ws_decay = reinterpret_cast<float *>(ws + pl.off_decay);
  }
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const unsigned gx = static_cast<unsigned>(blocks);
  if (pl.nseg > 1) {
    const hipError_t e = launch_var(a->dstate, false, dim3(gx, pl.nseg - 1), stream, p);
    if (e != hipSuccess) return hip_fail(e);
  }
  const hipError_t e = launch_var(a->dstate, true, dim3(gx, pl.nseg), stream, p);
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}
