// rms_norm.hip -- root-mean-square norm with the residual's addition or behind
// a gate, to io or to 8 bits (rms_norm_fwd), and its gradient (rms_norm_bwd).
//
// A workgroup takes a row, group by group.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_util.h"
#include "host_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct NormParams {
  const void *x, *z, *res, *dy, *ds;
  const float *w;
  void *rout, *out, *dx, *dres, *dz;
  uint8_t *codes;
  float *scales, *stat, *dw;
  int64_t rows, cols, group, xs, zs, rs, ros, os, cs, dys, dss, dxs, drs, dzs;
  float eps;
};

__device__ __forceinline__ float block_sum(float v, float *lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int k = 0; k < kThreads / 64; ++k) s += lds[k];
  return s;
}

// One code of a value: the hardware's rounding to e4m3, ties to even.
__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}
// The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8), and 1 / s.
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

// What is normalised at (row, column): MODE 0 x, 1 x + residual (RES its type), 2 x silu(z).
template <int IO, int MODE, int RES>
__device__ __forceinline__ float value_at(const NormParams &p, int64_t row, int64_t c) {
  const float x = load_io<IO>(p.x, row * p.xs + c);
  if constexpr (MODE == 1) return round_io<RES>(x + load_io<RES>(p.res, row * p.rs + c));
  if constexpr (MODE == 2) return x * silu_f(load_io<IO>(p.z, row * p.zs + c));
  return x;
}

template <int IO, int MODE, int RES>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormParams p) {
  __shared__ float lds[kThreads / 64];
  __shared__ float v[RMS_MAX_GROUP / kThreads][kThreads];
  __shared__ uint32_t top[RMS_MAX_GROUP / RMS_SCALE_BLOCK];
  const int64_t row = blockIdx.x, first = blockIdx.y * p.group;
  const int n = static_cast<int>(p.group), nb = (n + RMS_SCALE_BLOCK - 1) / RMS_SCALE_BLOCK;
  float sum = 0.0f;
  for (int k = threadIdx.x; k < n; k += kThreads) {
    const float q = value_at<IO, MODE, RES>(p, row, first + k);
    v[k / kThreads][threadIdx.x] = q;
    if constexpr (MODE == 1) store_one<RES>(p.rout, row * p.ros + first + k, q);
    sum = fmaf(q, q, sum);
  }
  for (int k = threadIdx.x; k < nb; k += kThreads) top[k] = 0;
  const float rstd = 1.0f / sqrtf(block_sum(sum, lds) / n + p.eps);
  for (int k = threadIdx.x; k < n; k += kThreads) {
    const float y = v[k / kThreads][threadIdx.x] * rstd * p.w[first + k];
    v[k / kThreads][threadIdx.x] = y;
    if (p.codes) atomicMax(&top[k / RMS_SCALE_BLOCK], __float_as_uint(y) & 0x7fffffffu);
    else store_one<IO>(p.out, row * p.os + first + k, y);
  }
  if (!p.codes) return;
  __syncthreads();
  for (int k = threadIdx.x; k < n; k += kThreads) {
    float inv;
    const float scale = e4m3_scale(top[k / RMS_SCALE_BLOCK], inv);
    p.codes[row * p.cs + first + k] = to_e4m3(v[k / kThreads][threadIdx.x] * inv);
    if (k % RMS_SCALE_BLOCK == 0)
      p.scales[row * ((p.cols + RMS_SCALE_BLOCK - 1) / RMS_SCALE_BLOCK) + (first + k) / RMS_SCALE_BLOCK] = scale;
  }
}

template <int IO, int XT, bool GATE>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormParams p) {
  __shared__ float lds[kThreads / 64];
  const int64_t row = blockIdx.x, first = blockIdx.y * p.group;
  const int n = static_cast<int>(p.group);
  float sum = 0.0f, dot = 0.0f;
  for (int k = threadIdx.x; k < n; k += kThreads) {
    float v = load_io<XT>(p.x, row * p.xs + first + k);
    if constexpr (GATE) v *= silu_f(load_io<IO>(p.z, row * p.zs + first + k));
    sum = fmaf(v, v, sum);
    dot = fmaf(v, load_io<IO>(p.dy, row * p.dys + first + k) * p.w[first + k], dot);
  }
  const float rstd = 1.0f / sqrtf(block_sum(sum, lds) / n + p.eps);
  const float mean = block_sum(dot, lds) * rstd / n;
  if (threadIdx.x == 0) p.stat[row * gridDim.y + blockIdx.y] = rstd;
  for (int k = threadIdx.x; k < n; k += kThreads) {
    const float x = load_io<XT>(p.x, row * p.xs + first + k);
    float gate = 1.0f, dgate = 0.0f;
    if constexpr (GATE) {
      const float z = load_io<IO>(p.z, row * p.zs + first + k), sg = fast_rcp(1.0f + fast_exp2(-z * kLog2e));
      gate = z * sg;
      dgate = sg * fmaf(z, 1.0f - sg, 1.0f);
    }
    const float dv = rstd * fmaf(-x * gate * rstd, mean, load_io<IO>(p.dy, row * p.dys + first + k) * p.w[first + k]);
    float dx = dv * gate;
    if (p.ds) dx += load_io<XT>(p.ds, row * p.dss + first + k);
    if (p.dres) store_one<XT>(p.dres, row * p.drs + first + k, dx);
    store_one<IO>(p.dx, row * p.dxs + first + k, dx);
    if constexpr (GATE) store_one<IO>(p.dz, row * p.dzs + first + k, dv * x * dgate);
  }
}

template <int IO, int XT, bool GATE>
__global__ void __launch_bounds__(64) norm_dweight_kernel(const NormParams p) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (c >= p.cols) return;
  double v = 0.0;
  for (int64_t row = 0; row < p.rows; ++row) {
    float x = load_io<XT>(p.x, row * p.xs + c);
    if constexpr (GATE) x *= silu_f(load_io<IO>(p.z, row * p.zs + c));
    v += x * p.stat[row * (p.cols / p.group) + c / p.group] * load_io<IO>(p.dy, row * p.dys + c);
  }
  p.dw[c] = static_cast<float>(v);
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

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int rms_norm_fwd(const rms_norm_args_t *a, void *stream_ptr) {
  const int st = rms_norm_fwd_validate(a);
  if (st != SSM_OK) return st;
  const int64_t groups = a->cols / a->group_size;
  if (groups > 65535 || !grid_fits(a->rows, kThreads)) return SSM_ERR_SHAPE;
  NormParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.z = a->z; p.zs = a->z_stride;
  p.res = a->residual; p.rs = a->residual_stride;
  p.rout = a->residual_out; p.ros = a->residual_out_stride;
  p.w = a->weight; p.out = a->out; p.os = a->out_stride;
  p.codes = static_cast<uint8_t *>(a->codes); p.cs = a->codes_stride; p.scales = a->scales;
  p.rows = a->rows; p.cols = a->cols; p.group = a->group_size; p.eps = a->eps;
  const dim3 grid(static_cast<unsigned>(a->rows), static_cast<unsigned>(groups));
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  return by_io(a->io_dtype, [&](auto io) {
    constexpr int IO = decltype(io)::value;
    if (a->z) hipLaunchKernelGGL((norm_fwd_kernel<IO, 2, IO>), grid, dim3(kThreads), 0, stream, p);
    else if (!a->residual) hipLaunchKernelGGL((norm_fwd_kernel<IO, 0, IO>), grid, dim3(kThreads), 0, stream, p);
    else if (a->residual_dtype == a->io_dtype) hipLaunchKernelGGL((norm_fwd_kernel<IO, 1, IO>), grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((norm_fwd_kernel<IO, 1, SSM_F32>), grid, dim3(kThreads), 0, stream, p);
  });
}

extern "C" int rms_norm_bwd_workspace_size(const rms_norm_bwd_args_t *a, size_t *bytes) {
  const int st = rms_norm_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = static_cast<size_t>(a->rows) * (a->cols / a->group_size) * sizeof(float);
  return SSM_OK;
}

extern "C" int rms_norm_bwd(const rms_norm_bwd_args_t *a, void *stream_ptr) {
  size_t need = 0;
  const int st = rms_norm_bwd_workspace_size(a, &need);
  if (st != SSM_OK) return st;
  const int64_t groups = a->cols / a->group_size;
  if (groups > 65535 || !grid_fits(a->rows, kThreads)) return SSM_ERR_SHAPE;
  if (!a->workspace || a->workspace_bytes < need) return SSM_ERR_WORKSPACE;
  NormParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.z = a->z; p.zs = a->z_stride;
  p.dy = a->dy; p.dys = a->dy_stride;
  p.ds = a->ds; p.dss = a->ds_stride;
  p.dx = a->dx; p.dxs = a->dx_stride;
  p.dres = a->dresidual; p.drs = a->dresidual_stride;
  p.dz = a->dz; p.dzs = a->dz_stride;
  p.w = a->weight; p.dw = a->dweight; p.stat = static_cast<float *>(a->workspace);
  p.rows = a->rows; p.cols = a->cols; p.group = a->group_size; p.eps = a->eps;
  const dim3 grid(static_cast<unsigned>(a->rows), static_cast<unsigned>(groups));
  const dim3 cols(static_cast<unsigned>((a->cols + 63) / 64));
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  return by_io(a->io_dtype, [&](auto io) {
    constexpr int IO = decltype(io)::value;
    auto both = [&](auto xt, auto gate) {
      constexpr int XT = decltype(xt)::value;
      constexpr bool GATE = decltype(gate)::value;
      hipLaunchKernelGGL((norm_bwd_kernel<IO, XT, GATE>), grid, dim3(kThreads), 0, stream, p);
      hipLaunchKernelGGL((norm_dweight_kernel<IO, XT, GATE>), cols, dim3(64), 0, stream, p);
    };
    if (a->z) both(io, std::true_type{});
    else if (a->x_dtype == a->io_dtype) both(io, std::false_type{});
    else both(std::integral_constant<int, SSM_F32>{}, std::false_type{});
  });
}
