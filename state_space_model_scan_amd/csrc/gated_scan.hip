// gated_scan.hip -- the gated linear recurrence over packed tokens
// (gated_scan_varlen_fwd), its gradient (gated_scan_varlen_bwd) and its
// single-token step (gated_scan_update).
//
// A thread walks a (sequence, channel) token by token.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gated_util.h"
#include "host_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kT = GATED_CHUNK;

struct GatedParams {
  const void *x, *r, *i, *dout;
  void *out, *dx, *dr, *di;
  const float *A, *rb, *ib, *h0, *dfin;
  float *state, *ckpt, *part, *dinit;
  const int32_t *cu, *seen, *slots;
  int64_t total, nseq, channels, nslots, xs, rs, is, os, dos, dxs, drs, dis;
};

struct Span {
  int64_t lo, hi;
};
__device__ __forceinline__ Span span_of(const GatedParams &p, int64_t s) {
  int64_t lo = p.cu[s], hi = p.cu[s + 1];
  lo = lo < 0 ? 0 : lo > p.total ? p.total : lo;
  hi = hi < lo ? lo : hi > p.total ? p.total : hi;
  return {lo, hi};
}

template <int IO>
__device__ __forceinline__ Gates token_gates(const GatedParams &p, int64_t t, int64_t c, float A, float rb, float ib) {
  return gates_of(load_io<IO>(p.r, t * p.rs + c) + rb, load_io<IO>(p.i, t * p.is + c) + ib, A);
}

template <int IO>
__global__ void __launch_bounds__(64) gated_fwd_kernel(const GatedParams p) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t s = blockIdx.y;
  const Span q = span_of(p, s);
  const int64_t slot = p.slots ? p.slots[s] : s;
  const bool cached = p.state && slot >= 0 && slot < p.nslots;
  const float A = p.A[c], rb = p.rb ? p.rb[c] : 0.0f, ib = p.ib ? p.ib[c] : 0.0f;
  float h = cached && p.seen && p.seen[s] > 0 ? p.state[slot * p.channels + c] : 0.0f;
  for (int64_t t = q.lo; t < q.hi; ++t) {
    if (p.ckpt && t % kT == 0) p.ckpt[t / kT * p.channels + c] = h;
    const Gates g = token_gates<IO>(p, t, c, A, rb, ib);
    h = fmaf(g.a, h, g.m * (g.iota * load_io<IO>(p.x, t * p.xs + c)));
    store_one<IO>(p.out, t * p.os + c, h);
  }
  if (cached && q.hi > q.lo) p.state[slot * p.channels + c] = h;
}

// Tokens of no sequence: kept states and gradients of 0.
template <int IO>
__global__ void __launch_bounds__(64) gated_rest_kernel(const GatedParams p) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t first = p.cu[0] < 0 ? 0 : p.cu[0], end = p.cu[p.nseq] < first ? first : p.cu[p.nseq];
  for (int64_t t = 0; t < p.total; t = t + 1 == first && end > first ? end : t + 1) {
    if (t >= first && t < end) continue;
    if (p.dx) {
      store_one<IO>(p.dx, t * p.dxs + c, 0.0f);
      store_one<IO>(p.dr, t * p.drs + c, 0.0f);
      store_one<IO>(p.di, t * p.dis + c, 0.0f);
    } else if (p.ckpt && t % kT == 0) {
      p.ckpt[t / kT * p.channels + c] = 0.0f;
    }
  }
}

template <int IO>
__global__ void __launch_bounds__(64) gated_bwd_kernel(const GatedParams p) {
  __shared__ float before[kT][64];
  const int lane = threadIdx.x;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  if (c >= p.channels) return;
  const int64_t s = blockIdx.y;
  const Span q = span_of(p, s);
  const float A = p.A[c], rb = p.rb ? p.rb[c] : 0.0f, ib = p.ib ? p.ib[c] : 0.0f;
  const float h0 = p.h0 ? p.h0[s * p.channels + c] : 0.0f;
  float come = p.dfin ? p.dfin[s * p.channels + c] : 0.0f, dA = 0.0f, drb = 0.0f, dib = 0.0f;
  for (int64_t k = (q.hi - 1) / kT; q.hi > q.lo && k >= q.lo / kT; --k) {
    const int64_t from = k * kT > q.lo ? k * kT : q.lo, to = (k + 1) * kT < q.hi ? (k + 1) * kT : q.hi;
    float h = from == q.lo ? h0 : p.ckpt[k * p.channels + c];
    for (int64_t t = from; t < to; ++t) {
      before[t - from][lane] = h;
      const Gates g = token_gates<IO>(p, t, c, A, rb, ib);
      h = fmaf(g.a, h, g.m * (g.iota * load_io<IO>(p.x, t * p.xs + c)));
    }
    for (int64_t t = to - 1; t >= from; --t) {
      const Gates g = token_gates<IO>(p, t, c, A, rb, ib);
      const float adj = load_io<IO>(p.dout, t * p.dos + c) + come;
      come = g.a * adj;
      const float x = load_io<IO>(p.x, t * p.xs + c), gated = g.iota * x;
      const float w = adj * g.rho * g.a * (before[t - from][lane] - g.a * g.inv_m * gated);
      const float dr = A * (1.0f - g.rho) * w, di = adj * g.m * gated * (1.0f - g.iota);
      dA += w;
      drb += dr;
      dib += di;
      store_one<IO>(p.dx, t * p.dxs + c, adj * g.m * g.iota);
      store_one<IO>(p.dr, t * p.drs + c, dr);
      store_one<IO>(p.di, t * p.dis + c, di);
    }
  }
  if (p.dinit) p.dinit[s * p.channels + c] = come;
  float *part = p.part + s * 3 * p.channels + c;
  part[0] = dA;
  part[p.channels] = drb;
  part[2 * p.channels] = dib;
}

__global__ void __launch_bounds__(64) gated_sum_kernel(const float *part, int64_t rows, int64_t channels, float *dA, float *drb,
                                                       float *dib) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (c >= channels) return;
  double v[3] = {0.0, 0.0, 0.0};
  for (int64_t k = 0; k < rows; ++k)
    for (int j = 0; j < 3; ++j) v[j] += part[(k * 3 + j) * channels + c];
  dA[c] = static_cast<float>(v[0]);
  if (drb) drb[c] = static_cast<float>(v[1]);
  if (dib) dib[c] = static_cast<float>(v[2]);
}

struct UpdateParams {
  const void *x, *r, *i;
  void *out;
  const float *A, *rb, *ib;
  float *state;
  const int32_t *seen, *slots;
  int64_t channels, nslots, xs, rs, is, os;
};

template <int IO>
__global__ void __launch_bounds__(64) gated_update_kernel(const UpdateParams p) {
  const int64_t c = static_cast<int64_t>(blockIdx.y) * 64 + threadIdx.x;
  if (c >= p.channels) return;
  const int64_t b = blockIdx.x;
  const int64_t slot = p.slots ? p.slots[b] : b;
  const bool cached = slot >= 0 && slot < p.nslots;
  const Gates g = gates_of(load_io<IO>(p.r, b * p.rs + c) + (p.rb ? p.rb[c] : 0.0f),
                           load_io<IO>(p.i, b * p.is + c) + (p.ib ? p.ib[c] : 0.0f), p.A[c]);
  float h = cached && p.seen && p.seen[b] > 0 ? p.state[slot * p.channels + c] : 0.0f;
  h = fmaf(g.a, h, g.m * (g.iota * load_io<IO>(p.x, b * p.xs + c)));
  store_one<IO>(p.out, b * p.os + c, h);
  if (cached) p.state[slot * p.channels + c] = h;
}

GatedParams gated_params(const gated_scan_varlen_args_t &a) {
  GatedParams p{};
  p.x = a.x; p.xs = a.x_stride;
  p.r = a.r; p.rs = a.r_stride;
  p.i = a.i; p.is = a.i_stride;
  p.A = a.A; p.rb = a.r_bias; p.ib = a.i_bias; p.cu = a.cu_seqlens;
  p.total = a.total; p.nseq = a.nseq; p.channels = a.channels;
  p.ckpt = a.checkpoints;
  return p;
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

extern "C" int gated_scan_varlen_fwd_workspace_size(const gated_scan_varlen_args_t *a, size_t *bytes) {
  const int st = gated_scan_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = 0;
  return SSM_OK;
}

extern "C" int gated_scan_varlen_fwd(const gated_scan_varlen_args_t *a, void *stream_ptr) {
  const int st = gated_scan_varlen_fwd_validate(a);
  if (st != SSM_OK) return st;
  if (a->nseq > 65535) return SSM_ERR_SHAPE;
  GatedParams p = gated_params(*a);
  p.out = a->out; p.os = a->out_stride;
  p.state = a->state; p.nslots = a->state_slots; p.seen = a->cache_seqlens; p.slots = a->slots;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const unsigned gx = static_cast<unsigned>((a->channels + 63) / 64);
  return by_io(a->io_dtype, [&](auto io) {
    constexpr int IO = decltype(io)::value;
    if (p.ckpt) hipLaunchKernelGGL((gated_rest_kernel<IO>), dim3(gx), dim3(64), 0, stream, p);
    hipLaunchKernelGGL((gated_fwd_kernel<IO>), dim3(gx, static_cast<unsigned>(p.nseq)), dim3(64), 0, stream, p);
  });
}

extern "C" int gated_scan_varlen_bwd_workspace_size(const gated_scan_varlen_bwd_args_t *a, size_t *bytes) {
  const int st = gated_scan_varlen_bwd_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = static_cast<size_t>(a->fwd.nseq) * 3 * a->fwd.channels * sizeof(float);
  return SSM_OK;
}

extern "C" int gated_scan_varlen_bwd(const gated_scan_varlen_bwd_args_t *a, void *stream_ptr) {
  size_t need = 0;
  const int st = gated_scan_varlen_bwd_workspace_size(a, &need);
  if (st != SSM_OK) return st;
  if (a->fwd.nseq > 65535) return SSM_ERR_SHAPE;
  if (!a->workspace || a->workspace_bytes < need) return SSM_ERR_WORKSPACE;
  GatedParams p = gated_params(a->fwd);
  p.dout = a->dout; p.dos = a->dout_stride;
  p.dx = a->dx; p.dxs = a->dx_stride;
  p.dr = a->dr; p.drs = a->dr_stride;
  p.di = a->di; p.dis = a->di_stride;
  p.h0 = a->initial_states; p.dfin = a->dfinal_states; p.dinit = a->dinitial_states;
  p.part = static_cast<float *>(a->workspace);
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const unsigned gx = static_cast<unsigned>((p.channels + 63) / 64);
  return by_io(a->fwd.io_dtype, [&](auto io) {
    constexpr int IO = decltype(io)::value;
    hipLaunchKernelGGL((gated_rest_kernel<IO>), dim3(gx), dim3(64), 0, stream, p);
    hipLaunchKernelGGL((gated_bwd_kernel<IO>), dim3(gx, static_cast<unsigned>(p.nseq)), dim3(64), 0, stream, p);
    hipLaunchKernelGGL(gated_sum_kernel, dim3(gx), dim3(64), 0, stream, p.part, p.nseq, p.channels, a->dA, a->dr_bias, a->di_bias);
  });
}

extern "C" int gated_scan_update(const gated_scan_update_args_t *a, void *stream_ptr) {
  const int st = gated_scan_update_validate(a);
  if (st != SSM_OK) return st;
  const int64_t gy = (a->channels + 63) / 64;
  if (gy > 65535 || !grid_fits(a->batch, 64)) return SSM_ERR_SHAPE;
  UpdateParams p{};
  p.x = a->x; p.xs = a->x_stride;
  p.r = a->r; p.rs = a->r_stride;
  p.i = a->i; p.is = a->i_stride;
  p.out = a->out; p.os = a->out_stride;
  p.A = a->A; p.rb = a->r_bias; p.ib = a->i_bias;
  p.state = a->state; p.nslots = a->state_slots; p.seen = a->cache_seqlens; p.slots = a->slots;
  p.channels = a->channels;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const dim3 grid(static_cast<unsigned>(a->batch), static_cast<unsigned>(gy));
  return by_io(a->io_dtype, [&](auto io) {
    hipLaunchKernelGGL((gated_update_kernel<decltype(io)::value>), grid, dim3(64), 0, stream, p);
  });
}
