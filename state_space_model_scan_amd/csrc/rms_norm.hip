// rms_norm.hip -- root-mean-square norm with the residual's addition or behind
// a gate, to io or to 8 bits (rms_norm_fwd), and its gradient (rms_norm_bwd).
//
// Both stream: every element is read once, held in registers, and written once.
// A group of columns is a unit of its own; L lanes take it (8 to 64 of a wave,
// or 2 to 8 whole waves), each K vectors of V neighbouring columns (16 bytes),
// as few lanes as K allows: then a wave has more loads in flight, fewer idle
// lanes and no barrier.  Vectors are read and written at any address: rows of
// 1003 elements have no other, and single elements took 20.6 us for 8192 of them
// with a residual.
//
// Measured on bf16 (us; bytes over time): 16384 x 5120 gated in eight groups 90
// (5.6 TB/s, a copy makes 5.1), 4100 x 2560 with a residual to 8 bits 16 (4.6), the
// gradient of 16384 x 2560 with the residual stream in fp32 128 (5.2): HBM.
//
// The gradient's workgroups walk the rows of their units, so that a lane's
// weight gradients stay in its registers; the workgroups' sums are added by a
// second launch, in a fixed order.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "column_sum.h"
#include "device_util.h"
#include "host_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kMaxThreads = 512;

struct NormParams {
  const void *x, *z, *res, *dy, *ds;
  const float *w;
  void *rout, *out, *dx, *dres, *dz;
  uint8_t *codes;
  float *scales, *part, *dw;
  int64_t rows, cols, xs, zs, rs, ros, os, cs, dys, dss, dxs, drs, dzs;
  int group, groups, lanes;   // lanes: of a unit, a power of two
  float eps;
};

// V neighbouring elements at any address of one, or the first `n` of them (the
// others 0).
template <int BYTES, int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Words {
  uint32_t w[BYTES / 4];
};
template <int IO, int V>
struct Vec {
  static constexpr int kSize = IO == 0 ? 4 : 2;
  using At = Words<V * kSize, kSize>;
  RawV<IO, V> r;
  template <bool TAIL>
  __device__ __forceinline__ void load(const void *p, int64_t i, int n) {
    if (!TAIL || n >= V) {
      const At q = *reinterpret_cast<const At *>(static_cast<const char *>(p) + i * kSize);
#pragma unroll
      for (int k = 0; k < RawV<IO, V>::kWords; ++k) r.w[k] = q.w[k];
    } else {
      r.load_elems(p, i, n);
    }
  }
  __device__ __forceinline__ float get(int k) const { return r.get(k); }
  __device__ __forceinline__ void zero() { r.zero(); }
};
template <int IO, int V, bool TAIL>
__device__ __forceinline__ void put(void *p, int64_t i, const float (&v)[V], int n) {
  using At = typename Vec<IO, V>::At;
  if (TAIL && n < V) {
    store_n<IO, V>(p, i, v, n, false);
    return;
  }
  At q;
  if constexpr (IO == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k) q.w[k] = __float_as_uint(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) q.w[k] = float_to_half_bits<IO>(v[2 * k]) | (float_to_half_bits<IO>(v[2 * k + 1]) << 16);
  }
  *reinterpret_cast<At *>(static_cast<char *>(p) + i * Vec<IO, V>::kSize) = q;
}

// Sum over a unit's lanes; more than a wave of them meet in LDS (`room`: a
// float for every wave of the workgroup), where every thread has to be there.
__device__ __forceinline__ float unit_sum(float v, int lanes, float *room) {
  const int in_wave = lanes < 64 ? lanes : 64;
  for (int o = 1; o < in_wave; o <<= 1) v += __shfl_xor(v, o);
  if (lanes <= 64) return v;
  const int wave = threadIdx.x >> 6, per = lanes >> 6, first = wave & ~(per - 1);
  if ((threadIdx.x & 63) == 0) room[wave] = v;
  __syncthreads();
  float s = 0.0f;
  for (int k = 0; k < per; ++k) s += room[first + k];
  return s;
}

// The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8), and 1 / s:
// a code times a power of two is exact in bf16, and against amax / 448 the
// coarser scale costs an e4m3 value none of its four significant bits.  At least
// 2^-100, which keeps every value a normal number.  NaN where amax is not finite.
__device__ __forceinline__ float e4m3_scale(uint32_t amax, float &inv) {
  if (amax >= 0x7f800000u) {
    inv = 0.0f;
    return __uint_as_float(0x7fc00000u);
  }
  int e = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < -100 ? -100 : e;
  inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

enum Mode { kPlain, kAdd, kGate };

// RES: the residual's type.  8 bits: QUANT.  TAIL: a unit's columns are no
// multiple of V.
template <int IO, int MODE, int RES, bool QUANT, bool TAIL, int K>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const NormParams p) {
  constexpr int V = IO == 0 ? 4 : 8;
  __shared__ float room[kMaxThreads / 64];
  const int lane = threadIdx.x & (p.lanes - 1);
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / p.lanes;
  const int64_t row = unit / p.groups;
  const int first = static_cast<int>(unit - row * p.groups) * p.group;
  const bool there = row < p.rows;

  Vec<IO, V> x[K];
  Vec<MODE == kAdd ? RES : IO, V> r[MODE == kPlain ? 1 : K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * p.lanes + lane) * V, n = p.group - c;
    if (there && n > 0) {
      x[k].template load<TAIL>(p.x, row * p.xs + first + c, n);
      if constexpr (MODE == kAdd) r[k].template load<TAIL>(p.res, row * p.rs + first + c, n);
      if constexpr (MODE == kGate) r[k].template load<TAIL>(p.z, row * p.zs + first + c, n);
    } else {
      x[k].zero();
      if constexpr (MODE != kPlain) r[k].zero();
    }
  }
  float v[K][V], sum = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float q = x[k].get(i);
      if constexpr (MODE == kAdd) q = round_io<RES>(q + r[k].get(i));
      if constexpr (MODE == kGate) q *= silu_f(r[k].get(i));
      v[k][i] = q;
      sum = fmaf(q, q, sum);
    }
    if constexpr (MODE == kAdd) {
      const int c = (k * p.lanes + lane) * V, n = p.group - c;
      if (there && n > 0) put<RES, V, TAIL>(p.rout, row * p.ros + first + c, v[k], n);
    }
  }
  sum = unit_sum(sum, p.lanes, room);
  const float rstd = 1.0f / sqrtf(sum / p.group + p.eps);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * p.lanes + lane) * V, n = p.group - c;
    const bool in = there && n > 0;
    Vec<0, V> w;
    if (in) w.template load<TAIL>(p.w, first + c, n);
    else w.zero();
#pragma unroll
    for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * rstd * w.get(i);
    if constexpr (!QUANT) {
      if (in) put<IO, V, TAIL>(p.out, row * p.os + first + c, v[k], n);
    } else {   // 128 / V neighbouring lanes hold a block
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t b = __float_as_uint(v[k][i]) & 0x7fffffffu;
        amax = in && (!TAIL || i < n) && b > amax ? b : amax;
      }
#pragma unroll
      for (int o = 1; o < RMS_SCALE_BLOCK / V; o <<= 1) {
        const uint32_t other = __shfl_xor(amax, o);
        amax = other > amax ? other : amax;
      }
      float inv;
      const float scale = e4m3_scale(amax, inv);
      if (!in) continue;
      Words<V, 1> q;
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const int h = __builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * i] * inv, v[k][4 * i + 1] * inv, 0, false);
        q.w[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * i + 2] * inv, v[k][4 * i + 3] * inv, h, true));
      }
      uint8_t *at = p.codes + row * p.cs + first + c;
      if (!TAIL || n >= V) {
        *reinterpret_cast<Words<V, 1> *>(at) = q;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < n) at[i] = static_cast<uint8_t>(q.w[i / 4] >> (8 * (i % 4)));
      }
      if (c % RMS_SCALE_BLOCK == 0)
        p.scales[row * ((p.cols + RMS_SCALE_BLOCK - 1) / RMS_SCALE_BLOCK) + (first + c) / RMS_SCALE_BLOCK] = scale;
    }
  }
}

// XT: x's type.  A workgroup's units are `blockDim.x / lanes` rows of one group
// of columns at a time; it walks the rows in steps of the whole grid.
template <int IO, int XT, bool GATE, bool TAIL, int K>
__global__ void __launch_bounds__(kMaxThreads, 2) norm_bwd_kernel(const NormParams p) {
  constexpr int V = IO == 0 ? 4 : 8;
  __shared__ float room[2][kMaxThreads / 64];
  extern __shared__ float sums[];
  const int lane = threadIdx.x & (p.lanes - 1), here = threadIdx.x / p.lanes, units = blockDim.x / p.lanes;
  const int first = blockIdx.y * p.group;
  float w[K][V], dw[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * p.lanes + lane) * V, n = p.group - c;
    Vec<0, V> q;
    if (n > 0) q.template load<TAIL>(p.w, first + c, n);
    else q.zero();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[k][i] = q.get(i);
      dw[k][i] = 0.0f;
    }
  }
  const float count = static_cast<float>(p.group);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * units; base < p.rows; base += static_cast<int64_t>(gridDim.x) * units) {
    const int64_t row = base + here;
    const bool there = row < p.rows;
    Vec<XT, V> x[K], ds[GATE ? 1 : K];
    Vec<IO, V> dy[K], z[GATE ? K : 1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.lanes + lane) * V, n = p.group - c;
      if (there && n > 0) {
        x[k].template load<TAIL>(p.x, row * p.xs + first + c, n);
        dy[k].template load<TAIL>(p.dy, row * p.dys + first + c, n);
        if constexpr (GATE) z[k].template load<TAIL>(p.z, row * p.zs + first + c, n);
        else if (p.ds) ds[k].template load<TAIL>(p.ds, row * p.dss + first + c, n);
        else ds[k].zero();
      } else {
        x[k].zero();
        dy[k].zero();
        if constexpr (GATE) z[k].zero();
        else ds[k].zero();
      }
    }
    float sum = 0.0f, dot = 0.0f, sg[GATE ? K : 1][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = x[k].get(i);
        if constexpr (GATE) {
          const float q = z[k].get(i);
          sg[k][i] = fast_rcp(1.0f + fast_exp2(-q * kLog2e));
          v *= q * sg[k][i];
        }
        sum = fmaf(v, v, sum);
        dot = fmaf(v, dy[k].get(i) * w[k][i], dot);
      }
    if (p.lanes > 64) __syncthreads();   // (the room's last readers are done)
    sum = unit_sum(sum, p.lanes, room[0]);
    dot = unit_sum(dot, p.lanes, room[1]);
    // 0 for a unit without a row: with eps = 0 its 1 / 0 would reach the weight's gradient, which its lanes share
    const float rstd = there ? 1.0f / sqrtf(sum / count + p.eps) : 0.0f;
    const float mean = dot * rstd / count;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.lanes + lane) * V, n = p.group - c;
      float dx[V], dz[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xv = x[k].get(i), g = dy[k].get(i);
        if constexpr (GATE) {
          const float q = z[k].get(i), s = sg[k][i], gate = q * s, hat = xv * gate * rstd;
          const float dv = rstd * fmaf(-hat, mean, g * w[k][i]);
          dw[k][i] = fmaf(g, hat, dw[k][i]);
          dx[i] = dv * gate;
          dz[i] = dv * xv * (s * fmaf(q, 1.0f - s, 1.0f));
        } else {
          const float hat = xv * rstd;
          dw[k][i] = fmaf(g, hat, dw[k][i]);
          dx[i] = fmaf(rstd, fmaf(-hat, mean, g * w[k][i]), ds[k].get(i));
        }
      }
      if (!there || n <= 0) continue;
      put<IO, V, TAIL>(p.dx, row * p.dxs + first + c, dx, n);
      if constexpr (GATE) put<IO, V, TAIL>(p.dz, row * p.dzs + first + c, dz, n);
      else if (p.dres) put<XT, V, TAIL>(p.dres, row * p.drs + first + c, dx, n);
    }
  }
  // the units' sums, in order and in 64 bits
  if (units > 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) sums[(k * V + i) * blockDim.x + threadIdx.x] = dw[k][i];
    __syncthreads();
    for (int at = here; at < K * V; at += units) {   // (a unit's lanes take an element of every lane)
      double s = 0.0;
      for (int u = 0; u < units; ++u) s += sums[at * blockDim.x + u * p.lanes + lane];
      const int c = (at / V * p.lanes + lane) * V + at % V;
      if (c < p.group) p.part[static_cast<int64_t>(blockIdx.x) * p.cols + first + c] = static_cast<float>(s);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * p.lanes + lane) * V, n = p.group - c;
    if (n > 0) put<0, V, TAIL>(p.part, static_cast<int64_t>(blockIdx.x) * p.cols + first + c, dw[k], n);
  }
}

// The workgroups' sums, added.
__global__ void __launch_bounds__(kSumThreads) norm_sum_kernel(const float *part, float *dw, int64_t rows, int64_t cols) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const double v = column_sum(part, rows, cols, col);
  if (threadIdx.x < 32 && col < cols) dw[col] = static_cast<float>(v);
}

// Vectors of a lane: of 8 columns of 16 bits, or 4 of 32.
constexpr int kWideK[] = {1, 2, 3, 5};
constexpr int kFloatK[] = {1, 2, 3, 5, 8};
using WideK = std::integer_sequence<int, 1, 2, 3, 5>;
using FloatK = std::integer_sequence<int, 1, 2, 3, 5, 8>;
static_assert(kMaxThreads * 5 * 8 >= RMS_MAX_GROUP && kMaxThreads * 8 * 4 >= RMS_MAX_GROUP,
              "the largest group fits a workgroup's registers");

// How a call's units are laid on lanes.
struct Lay {
  int v, k, lanes, threads;
  bool tail;
};
template <int N>
Lay lay_of(int64_t group, int v, const int (&ks)[N], int least, int most_k) {
  Lay l{};
  const int64_t vecs = (group + v - 1) / v;
  l.v = v;
  l.tail = group % v != 0;
  l.lanes = least;
  while (l.lanes < kMaxThreads && (vecs + l.lanes - 1) / l.lanes > most_k) l.lanes *= 2;
  for (int i = N - 1; i >= 0; --i)
    if ((vecs + l.lanes - 1) / l.lanes <= ks[i]) l.k = ks[i];
  l.threads = l.lanes > 256 ? l.lanes : 256;
  return l;
}
// `columns`: of a lane, where the largest groups do not take more.
Lay lay_of(int32_t io, int64_t group, int least, int columns) {
  return io == SSM_F32 ? lay_of(group, 4, kFloatK, least, columns / 4) : lay_of(group, 8, kWideK, least, columns / 8);
}

template <typename F>
int by_io(int32_t io, F &&launch) {
  using std::integral_constant;
  if (io == SSM_BF16) launch(integral_constant<int, SSM_BF16>{});
  else if (io == SSM_F16) launch(integral_constant<int, SSM_F16>{});
  else launch(integral_constant<int, SSM_F32>{});
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}
template <int... Ks, typename F>
void by_k(std::integer_sequence<int, Ks...>, int k, F &&launch) {
  ((k == Ks ? launch(std::integral_constant<int, Ks>{}) : void()), ...);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int rms_norm_fwd(const rms_norm_args_t *a, void *stream_ptr) {
  const int st = rms_norm_fwd_validate(a);
  if (st != SSM_OK) return st;
  const int32_t io = a->io_dtype;
  const int64_t groups = a->cols / a->group_size;
  // 8 bits: a block of 128 columns in neighbouring lanes of a wave.  Columns of a lane, 40 / 24 / 16 / 8 (us): bf16 16384 x 2560 with a residual 64.3
  // / 61.0 / 60.5 / 62.5, gated 16384 x 5120 in eight groups 92 / 89 / 97 / 117; fp32
  // 8192 x 2560 63.3 / 63.4 / 60.0 / 62.6.
  const Lay l = lay_of(io, a->group_size, !a->codes ? 8 : RMS_SCALE_BLOCK / (io == SSM_F32 ? 4 : 8), io == SSM_F32 ? 16 : 24);
  const int64_t units = l.threads / l.lanes, blocks = (a->rows * groups + units - 1) / units;
  if (!grid_fits(blocks, l.threads)) return SSM_ERR_SHAPE;
  NormParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.z = a->z; p.zs = a->z_stride;
  p.res = a->residual; p.rs = a->residual_stride;
  p.rout = a->residual_out; p.ros = a->residual_out_stride;
  p.w = a->weight; p.out = a->out; p.os = a->out_stride;
  p.codes = static_cast<uint8_t *>(a->codes); p.cs = a->codes_stride; p.scales = a->scales;
  p.rows = a->rows; p.cols = a->cols; p.eps = a->eps;
  p.group = static_cast<int>(a->group_size); p.groups = static_cast<int>(groups); p.lanes = l.lanes;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const dim3 grid(static_cast<unsigned>(blocks)), block(l.threads);
  return by_io(io, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    auto go = [&](auto mode, auto res, auto quant) {
      constexpr int MODE = decltype(mode)::value, RES = decltype(res)::value;
      constexpr bool QUANT = decltype(quant)::value;
      by_k(std::conditional_t<IO == 0, FloatK, WideK>{}, l.k, [&](auto k) {
        constexpr int K = decltype(k)::value;
        if (l.tail) hipLaunchKernelGGL((norm_fwd_kernel<IO, MODE, RES, QUANT, true, K>), grid, block, 0, stream, p);
        else hipLaunchKernelGGL((norm_fwd_kernel<IO, MODE, RES, QUANT, false, K>), grid, block, 0, stream, p);
      });
    };
    auto quant = [&](auto mode, auto res) {
      if (a->codes) go(mode, res, std::true_type{});
      else go(mode, res, std::false_type{});
    };
    if (a->z) quant(std::integral_constant<int, kGate>{}, type);
    else if (!a->residual) quant(std::integral_constant<int, kPlain>{}, type);
    else if (a->residual_dtype == io) quant(std::integral_constant<int, kAdd>{}, type);
    else quant(std::integral_constant<int, kAdd>{}, std::integral_constant<int, SSM_F32>{});
  });
}

namespace {

struct BwdPlan {
  Lay lay;
  int64_t blocks, groups;   // blocks: workgroups that share a group's rows
};
int64_t ceil_div(int64_t n, int64_t by) { return (n + by - 1) / by; }
// Two workgroups a compute unit walk many rows best; up to three passes over
// the rows four of them, as then a pass is what counts (us, two / four): 16384 x
// 2560 133 / 138, gated 16384 x 5120 in eight groups 172 / 178, but 1500 x 1001 in
// seven 16.5 / 14.0.  A call of a few passes of one workgroup takes one, which
// needs no second launch.
// A lane adds the weight gradient's terms of at most kLaneRows rows one after
// another in fp32, the rest is added in 64 bits: more rows take as many times the
// workgroups (us, without the limit / with it: 140000 x 2560 695 / 441, 131072 x 5120
// gated in groups of 80 2514 / 2231, 16384 x 5120 in groups of 8 777 / 544).
constexpr int64_t kLaneRows = 256;
BwdPlan bwd_plan(const rms_norm_bwd_args_t *a) {
  BwdPlan b{};
  b.groups = a->cols / a->group_size;
  // (columns of a lane: gated 16384 x 5120 in eight groups 172 us with 24, 218 with
  // 16, 645 with 40, which do not fit the registers; 16384 x 2560 129 with 16, 133
  // with 24, 155 with 40)
  b.lay = lay_of(a->io_dtype, a->group_size, 8, a->z ? 24 : 16);
  const int64_t units = b.lay.threads / b.lay.lanes, passes = (a->rows + units - 1) / units, cus = cu_count_cached();
  const int64_t few = ceil_div(4 * cus, b.groups);
  b.blocks = passes <= 4 ? 1 : passes > 3 * few ? ceil_div(2 * cus, b.groups) : passes < few ? passes : few;
  b.blocks *= ceil_div(passes, kLaneRows * b.blocks);
  return b;
}

}  // namespace

extern "C" int rms_norm_bwd_workspace_size(const rms_norm_bwd_args_t *a, size_t *bytes) {
  const int st = rms_norm_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  const BwdPlan b = bwd_plan(a);
  *bytes = b.blocks == 1 ? 0 : static_cast<size_t>(b.blocks) * a->cols * sizeof(float);
  return SSM_OK;
}

extern "C" int rms_norm_bwd(const rms_norm_bwd_args_t *a, void *stream_ptr) {
  size_t need = 0;
  const int st = rms_norm_bwd_workspace_size(a, &need);
  if (st != SSM_OK) return st;
  if (need && (!a->workspace || a->workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  if (need && reinterpret_cast<uintptr_t>(a->workspace) % alignof(float) != 0) return SSM_ERR_UNSUPPORTED;
  const BwdPlan b = bwd_plan(a);
  NormParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.z = a->z; p.zs = a->z_stride;
  p.dy = a->dy; p.dys = a->dy_stride;
  p.ds = a->ds; p.dss = a->ds_stride;
  p.dx = a->dx; p.dxs = a->dx_stride;
  p.dres = a->dresidual; p.drs = a->dresidual_stride;
  p.dz = a->dz; p.dzs = a->dz_stride;
  p.w = a->weight; p.part = b.blocks == 1 ? a->dweight : static_cast<float *>(a->workspace);
  p.rows = a->rows; p.cols = a->cols; p.eps = a->eps;
  p.group = static_cast<int>(a->group_size); p.groups = static_cast<int>(b.groups); p.lanes = b.lay.lanes;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  if (!grid_fits(b.blocks * b.groups, b.lay.threads)) return SSM_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>(b.blocks), static_cast<unsigned>(b.groups)), block(b.lay.threads);
  const size_t lds = b.lay.threads > b.lay.lanes ? static_cast<size_t>(b.lay.threads) * b.lay.k * b.lay.v * sizeof(float) : 0;
  return by_io(a->io_dtype, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    auto go = [&](auto xt, auto gate) {
      constexpr int XT = decltype(xt)::value;
      constexpr bool GATE = decltype(gate)::value;
      by_k(std::conditional_t<IO == 0, FloatK, WideK>{}, b.lay.k, [&](auto k) {
        constexpr int K = decltype(k)::value;
        if (b.lay.tail) hipLaunchKernelGGL((norm_bwd_kernel<IO, XT, GATE, true, K>), grid, block, lds, stream, p);
        else hipLaunchKernelGGL((norm_bwd_kernel<IO, XT, GATE, false, K>), grid, block, lds, stream, p);
      });
    };
    if (a->z) go(type, std::true_type{});
    else if (a->x_dtype == a->io_dtype) go(type, std::false_type{});
    else go(std::integral_constant<int, SSM_F32>{}, std::false_type{});
    if (b.blocks == 1) return;
    hipLaunchKernelGGL(norm_sum_kernel, dim3(static_cast<unsigned>((p.cols + 31) / 32)), dim3(kSumThreads), 0, stream, p.part, a->dweight,
                       b.blocks, p.cols);
  });
}
