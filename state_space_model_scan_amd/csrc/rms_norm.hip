// rms_norm.hip -- root-mean-square norm with the residual's addition or behind
// a gate, to io or to 8 bits (rms_norm_fwd), and its gradient (rms_norm_bwd).
//
// Both stream: every element is read once, held in registers, and written once.
// A group of columns is a unit of its own; L lanes take it (16 to 64 of a wave,
// or 2 to 8 whole waves), each K vectors of V neighbouring columns (16 bytes,
// or one element where rows are odd or not aligned), as few lanes as K allows:
// then a wave has more loads in flight, fewer idle lanes and no barrier.
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

// V elements of a type, 16 bytes of them (or 8 of 16 bits beside 8 of 32, in
// two loads), or one.
template <int IO, int V>
struct Vec {
  RawV<IO, V> r;
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
template <int IO, int V>
__device__ __forceinline__ void put(void *p, int64_t i, const float (&v)[V]) {
  if constexpr (V == 1) store_one<IO>(p, i, v[0]);
  else store_n<IO, V>(p, i, v, V, true);
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

// RES: the residual's type.  8 bits: QUANT.
template <int IO, int MODE, int RES, bool QUANT, int V, int K>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const NormParams p) {
  __shared__ float room[kMaxThreads / 64];
  __shared__ uint32_t top[QUANT && V == 1 ? RMS_MAX_GROUP / RMS_SCALE_BLOCK : 1];
  const int lane = threadIdx.x & (p.lanes - 1);
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / p.lanes;
  const int64_t row = unit / p.groups;
  const int first = static_cast<int>(unit - row * p.groups) * p.group;
  const bool there = row < p.rows;

  Vec<IO, V> x[K];
  Vec<MODE == kAdd ? RES : IO, V> r[MODE == kPlain ? 1 : K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * p.lanes + lane) * V;
    if (there && c < p.group) {
      x[k].load(p.x, row * p.xs + first + c);
      if constexpr (MODE == kAdd) r[k].load(p.res, row * p.rs + first + c);
      if constexpr (MODE == kGate) r[k].load(p.z, row * p.zs + first + c);
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
      const int c = (k * p.lanes + lane) * V;
      if (there && c < p.group) put<RES, V>(p.rout, row * p.ros + first + c, v[k]);
    }
  }
  sum = unit_sum(sum, p.lanes, room);
  const float rstd = 1.0f / sqrtf(sum / p.group + p.eps);
  if constexpr (!QUANT) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.lanes + lane) * V;
      if (!there || c >= p.group) continue;
      Vec<0, V> w;
      w.load(p.w, first + c);
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = v[k][i] * rstd * w.get(i);
      put<IO, V>(p.out, row * p.os + first + c, y);
    }
  } else {
    const int64_t blocks = (p.cols + RMS_SCALE_BLOCK - 1) / RMS_SCALE_BLOCK;
    if constexpr (V == 1) {   // a block's columns are spread over its unit's lanes: its largest through LDS (units of a wave or more: one a workgroup)
      for (int k = threadIdx.x; k < RMS_MAX_GROUP / RMS_SCALE_BLOCK; k += blockDim.x) top[k] = 0;
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.lanes + lane) * V;
      const bool in = there && c < p.group;
      uint32_t amax = 0;
      if (in) {
        Vec<0, V> w;
        w.load(p.w, first + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[k][i] *= rstd * w.get(i);
          const uint32_t b = __float_as_uint(v[k][i]) & 0x7fffffffu;
          amax = b > amax ? b : amax;
        }
      }
      if constexpr (V == 1) {
        if (in) atomicMax(&top[c / RMS_SCALE_BLOCK], amax);
      } else {   // 128 / V neighbouring lanes hold a block
#pragma unroll
        for (int o = 1; o < RMS_SCALE_BLOCK / V; o <<= 1) {
          const uint32_t other = __shfl_xor(amax, o);
          amax = other > amax ? other : amax;
        }
        float inv;
        const float scale = e4m3_scale(amax, inv);
        if (in) {
          uint32_t w[V / 4];
#pragma unroll
          for (int i = 0; i < V / 4; ++i) {
            int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * i] * inv, v[k][4 * i + 1] * inv, 0, false);
            w[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[k][4 * i + 2] * inv, v[k][4 * i + 3] * inv, q, true));
          }
          uint8_t *at = p.codes + row * p.cs + first + c;
          if constexpr (V == 8) *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint32_t *>(at) = w[0];
          if (c % RMS_SCALE_BLOCK == 0) p.scales[row * blocks + (first + c) / RMS_SCALE_BLOCK] = scale;
        }
      }
    }
    if constexpr (V == 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = k * p.lanes + lane;
        if (!there || c >= p.group) continue;
        float inv;
        const float scale = e4m3_scale(top[c / RMS_SCALE_BLOCK], inv), q = v[k][0] * inv;
        p.codes[row * p.cs + first + c] = static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false));
        if (c % RMS_SCALE_BLOCK == 0) p.scales[row * blocks + (first + c) / RMS_SCALE_BLOCK] = scale;
      }
    }
  }
}

// XT: x's type.  A workgroup's units are `blockDim.x / lanes` rows of one group
// of columns at a time; it walks the rows in steps of the whole grid.
template <int IO, int XT, bool GATE, int V, int K>
__global__ void __launch_bounds__(kMaxThreads, 2) norm_bwd_kernel(const NormParams p) {
  __shared__ float room[2][kMaxThreads / 64];
  extern __shared__ float sums[];
  const int lane = threadIdx.x & (p.lanes - 1), here = threadIdx.x / p.lanes, units = blockDim.x / p.lanes;
  const int first = blockIdx.y * p.group;
  float w[K][V], dw[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * p.lanes + lane) * V;
    Vec<0, V> q;
    if (c < p.group) q.load(p.w, first + c);
    else q.zero();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[k][i] = q.get(i);
      dw[k][i] = 0.0f;
    }
  }
  const float n = static_cast<float>(p.group);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * units; base < p.rows; base += static_cast<int64_t>(gridDim.x) * units) {
    const int64_t row = base + here;
    const bool there = row < p.rows;
    Vec<XT, V> x[K], ds[GATE ? 1 : K];
    Vec<IO, V> dy[K], z[GATE ? K : 1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.lanes + lane) * V;
      if (there && c < p.group) {
        x[k].load(p.x, row * p.xs + first + c);
        dy[k].load(p.dy, row * p.dys + first + c);
        if constexpr (GATE) z[k].load(p.z, row * p.zs + first + c);
        else if (p.ds) ds[k].load(p.ds, row * p.dss + first + c);
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
    const float rstd = 1.0f / sqrtf(sum / n + p.eps);
    const float mean = dot * rstd / n;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * p.lanes + lane) * V;
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
      if (!there || c >= p.group) continue;
      put<IO, V>(p.dx, row * p.dxs + first + c, dx);
      if constexpr (GATE) put<IO, V>(p.dz, row * p.dzs + first + c, dz);
      else if (p.dres) put<XT, V>(p.dres, row * p.drs + first + c, dx);
    }
  }
  // the units' sums, in order
  if (units > 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) sums[(k * V + i) * blockDim.x + threadIdx.x] = dw[k][i];
    __syncthreads();
    for (int at = here; at < K * V; at += units) {   // (a unit's lanes take an element of every lane)
      float s = 0.0f;
      for (int u = 0; u < units; ++u) s += sums[at * blockDim.x + u * p.lanes + lane];
      const int c = (at / V * p.lanes + lane) * V + at % V;
      if (c < p.group) p.part[static_cast<int64_t>(blockIdx.x) * p.cols + first + c] = s;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * p.lanes + lane) * V;
    if (c < p.group) put<0, V>(p.part, static_cast<int64_t>(blockIdx.x) * p.cols + first + c, dw[k]);
  }
}

// The workgroups' sums, added.
__global__ void __launch_bounds__(kSumThreads) norm_sum_kernel(const float *part, float *dw, int64_t rows, int64_t cols) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const double v = column_sum(part, rows, cols, col);
  if (threadIdx.x < 32 && col < cols) dw[col] = static_cast<float>(v);
}

// Vectors of a lane: of 8 columns of 16 bits or 4 of 32, and of single columns.
constexpr int kVecK[] = {1, 2, 3, 5};
constexpr int kVec4K[] = {1, 2, 3, 5, 8};
constexpr int kOneK[] = {4, 16, 32};
using VecK = std::integer_sequence<int, 1, 2, 3, 5>;
using Vec4K = std::integer_sequence<int, 1, 2, 3, 5, 8>;
using OneK = std::integer_sequence<int, 4, 16, 32>;
static_assert(kMaxThreads * 5 * 8 >= RMS_MAX_GROUP && kMaxThreads * 8 * 4 >= RMS_MAX_GROUP && kMaxThreads * 32 >= RMS_MAX_GROUP,
              "the largest group fits a workgroup's registers");

// How a call's units are laid on lanes: K vectors of V columns at most a lane.
struct Lay {
  int k, lanes, threads;
};
template <int N>
Lay lay_of(int64_t group, int v, const int (&ks)[N], int least, int most_k) {
  Lay l{};
  const int64_t vecs = (group + v - 1) / v;
  l.lanes = least;
  if (most_k > ks[N - 1]) most_k = ks[N - 1];
  while (l.lanes < kMaxThreads && (vecs + l.lanes - 1) / l.lanes > most_k) l.lanes *= 2;
  for (int i = N - 1; i >= 0; --i)
    if ((vecs + l.lanes - 1) / l.lanes <= ks[i]) l.k = ks[i];
  l.threads = l.lanes > 256 ? l.lanes : 256;
  return l;
}
// `columns`: of a lane, where the largest groups do not take more.
Lay lay_of(bool vec, int32_t io, int64_t group, int least, int columns) {
  if (!vec) return lay_of(group, 1, kOneK, least, columns > 16 ? 16 : 4);
  return io == SSM_F32 ? lay_of(group, 4, kVec4K, least, columns / 4) : lay_of(group, 8, kVecK, least, columns / 8);
}

bool wide(int32_t type, const void *p, int64_t stride, int v) {
  const int64_t bytes = type == SSM_F32 ? 4 : 2;
  const uintptr_t step = static_cast<uintptr_t>(v * bytes > 16 ? 16 : v * bytes);
  return stride % v == 0 && reinterpret_cast<uintptr_t>(p) % step == 0;
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
  const int v = io == SSM_F32 ? 4 : 8;
  const bool vec = a->group_size % v == 0 && wide(io, a->x, a->x_stride, v) && (!a->z || wide(io, a->z, a->z_stride, v)) &&
                   (!a->residual || (wide(a->residual_dtype, a->residual, a->residual_stride, v) &&
                                     wide(a->residual_dtype, a->residual_out, a->residual_out_stride, v))) &&
                   (!a->out || wide(io, a->out, a->out_stride, v)) && aligned16(a->weight) &&
                   (!a->codes || (a->codes_stride % v == 0 && reinterpret_cast<uintptr_t>(a->codes) % v == 0));
  const int64_t groups = a->cols / a->group_size;
  // (8 bits: a block of 128 columns in neighbouring lanes, or a workgroup a unit)
  const Lay l = lay_of(vec, io, a->group_size, !a->codes ? 8 : vec ? RMS_SCALE_BLOCK / v : 256, 40);
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
    constexpr int V = IO == 0 ? 4 : 8;
    auto go = [&](auto mode, auto res, auto quant) {
      constexpr int MODE = decltype(mode)::value, RES = decltype(res)::value;
      constexpr bool QUANT = decltype(quant)::value;
      if (vec)
        by_k(std::conditional_t<IO == 0, Vec4K, VecK>{}, l.k, [&](auto k) {
          hipLaunchKernelGGL((norm_fwd_kernel<IO, MODE, RES, QUANT, V, decltype(k)::value>), grid, block, 0, stream, p);
        });
      else
        by_k(OneK{}, l.k, [&](auto k) {
          hipLaunchKernelGGL((norm_fwd_kernel<IO, MODE, RES, QUANT, 1, decltype(k)::value>), grid, block, 0, stream, p);
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
  bool vec;
  Lay lay;
  int64_t blocks, groups;   // blocks: workgroups that share a group's rows
};
// The workspace's size goes by the sizes alone; a call whose strides allow no
// vectors takes another lay with as many blocks or fewer.
int64_t most_blocks(int64_t rows, int64_t groups) {
  const int64_t want = (4 * static_cast<int64_t>(cu_count_cached()) + groups - 1) / groups;
  return want < rows ? want : rows;
}
BwdPlan bwd_plan(const rms_norm_bwd_args_t *a) {
  BwdPlan b{};
  const int32_t io = a->io_dtype, xt = a->x_dtype;
  const int v = io == SSM_F32 ? 4 : 8;
  b.vec = a->group_size % v == 0 && wide(xt, a->x, a->x_stride, v) && wide(io, a->dy, a->dy_stride, v) &&
          wide(io, a->dx, a->dx_stride, v) && (!a->z || (wide(io, a->z, a->z_stride, v) && wide(io, a->dz, a->dz_stride, v))) &&
          (!a->ds || wide(xt, a->ds, a->ds_stride, v)) && (!a->dresidual || wide(xt, a->dresidual, a->dresidual_stride, v)) &&
          aligned16(a->weight);
  b.groups = a->cols / a->group_size;
  b.lay = lay_of(b.vec, io, a->group_size, 8, a->z ? 16 : 24);
  const int64_t units = b.lay.threads / b.lay.lanes, need = (a->rows + units - 1) / units, most = most_blocks(a->rows, b.groups);
  b.blocks = need < most ? need : most;
  return b;
}

}  // namespace

extern "C" int rms_norm_bwd_workspace_size(const rms_norm_bwd_args_t *a, size_t *bytes) {
  const int st = rms_norm_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = static_cast<size_t>(most_blocks(a->rows, a->cols / a->group_size)) * a->cols * sizeof(float);
  return SSM_OK;
}

extern "C" int rms_norm_bwd(const rms_norm_bwd_args_t *a, void *stream_ptr) {
  size_t need = 0;
  const int st = rms_norm_bwd_workspace_size(a, &need);
  if (st != SSM_OK) return st;
  if (!a->workspace || a->workspace_bytes < need) return SSM_ERR_WORKSPACE;
  const BwdPlan b = bwd_plan(a);
  if (b.groups > 65535) return SSM_ERR_SHAPE;
  NormParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.z = a->z; p.zs = a->z_stride;
  p.dy = a->dy; p.dys = a->dy_stride;
  p.ds = a->ds; p.dss = a->ds_stride;
  p.dx = a->dx; p.dxs = a->dx_stride;
  p.dres = a->dresidual; p.drs = a->dresidual_stride;
  p.dz = a->dz; p.dzs = a->dz_stride;
  p.w = a->weight; p.part = static_cast<float *>(a->workspace);
  p.rows = a->rows; p.cols = a->cols; p.eps = a->eps;
  p.group = static_cast<int>(a->group_size); p.groups = static_cast<int>(b.groups); p.lanes = b.lay.lanes;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const dim3 grid(static_cast<unsigned>(b.blocks), static_cast<unsigned>(b.groups)), block(b.lay.threads);
  const int v = !b.vec ? 1 : a->io_dtype == SSM_F32 ? 4 : 8;
  const size_t lds = b.lay.threads > b.lay.lanes ? static_cast<size_t>(b.lay.threads) * b.lay.k * v * sizeof(float) : 0;
  return by_io(a->io_dtype, [&](auto type) {
    constexpr int IO = decltype(type)::value;
    constexpr int V = IO == 0 ? 4 : 8;
    auto go = [&](auto xt, auto gate) {
      constexpr int XT = decltype(xt)::value;
      constexpr bool GATE = decltype(gate)::value;
      if (b.vec)
        by_k(std::conditional_t<IO == 0, Vec4K, VecK>{}, b.lay.k, [&](auto k) {
          hipLaunchKernelGGL((norm_bwd_kernel<IO, XT, GATE, V, decltype(k)::value>), grid, block, lds, stream, p);
        });
      else
        by_k(OneK{}, b.lay.k, [&](auto k) {
          hipLaunchKernelGGL((norm_bwd_kernel<IO, XT, GATE, 1, decltype(k)::value>), grid, block, lds, stream, p);
        });
    };
    if (a->z) go(type, std::true_type{});
    else if (a->x_dtype == a->io_dtype) go(type, std::false_type{});
    else go(std::integral_constant<int, SSM_F32>{}, std::false_type{});
    hipLaunchKernelGGL(norm_sum_kernel, dim3(static_cast<unsigned>((p.cols + 31) / 32)), dim3(kSumThreads), 0, stream, p.part, a->dweight,
                       b.blocks, p.cols);
  });
}
