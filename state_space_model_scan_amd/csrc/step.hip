// step.hip -- one token of a Mamba-2 mixer (conv1d_ssd_update): the short
// convolution against a ring of earlier inputs and the state update, in one
// launch.
//
// The call reads and writes every request's fp32 state once (32 KB a head at
// dstate 128) and little else, so it is bound by HBM; with one request it is
// bound by latency.  A workgroup takes `rows` of a head's 64 channels for one
// request: its part of the state is loaded into registers first (16 bytes a
// lane and row, non-temporal: it passes through once), and while those loads
// are in flight the convolution of the head's channels and of its group's B
// and C (again for every head: 4 products a channel) is formed in LDS.  B's
// and C's ring entries are read by every head's workgroup and written by the
// group's first one.  That needs no order between them, because the ring has
// at least `width` entries: the new input goes to an entry that no workgroup
// reads.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_util.h"
#include "host_util.h"
#include "ssmscan.h"

namespace ssm {
namespace {

constexpr int kW = SSM_CONV_WIDTH;
constexpr int kP = SSD_HEADDIM;

struct StepParams {
  const void *xBC, *dt, *z;
  const float *A, *w, *wb, *D, *dt_bias;
  void *ring, *out;
  float *state;
  const int32_t *seen, *slots;
  int64_t nheads, ngroups, xs, dts, zs, os, nslots;
  uint32_t per_group, ring_len;
  int silu, softplus, dt_limit, D_per_channel;
  float dt_min, dt_max;
};

// sum over the 2^k neighbouring lanes of a row
template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int IO, int N, int ROWS>
__global__ void __launch_bounds__(256) step_kernel(const StepParams p) {
  constexpr int LPR = N / 4;             // lanes of a state row
  constexpr int AT_ONCE = 256 / LPR;     // rows of a pass
  constexpr int PASSES = ROWS / AT_ONCE > 0 ? ROWS / AT_ONCE : 1;
  __shared__ __attribute__((aligned(16))) float su[ROWS + 2 * N];   // act(conv): x rows, B, C
  typedef float f4 __attribute__((ext_vector_type(4)));
  const int tid = threadIdx.x;
  const int h = blockIdx.x, row0 = blockIdx.y * ROWS;
  const int64_t b = blockIdx.z;
  const uint32_t g = static_cast<uint32_t>(h) / p.per_group;
  int64_t slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.nslots) slot = -1;
  int32_t seen = p.seen ? p.seen[b] : 0;
  if (seen < 0 || slot < 0) seen = 0;

  // ---- this workgroup's part of the state
  const int r = tid / LPR, n0 = (tid % LPR) * 4;
  float *srow = p.state + ((slot < 0 ? 0 : slot) * p.nheads + h) * kP * N + (row0 + r) * N + n0;
  f4 st[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    if (seen > 0 && r + i * AT_ONCE < ROWS)
      st[i] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(srow + i * AT_ONCE * N));
    else
      st[i] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
  }

  // ---- the convolution of x rows, B and C
  const int64_t hp = p.nheads * kP, channels = hp + 2 * p.ngroups * N;
  for (int i = tid; i < ROWS + 2 * N; i += 256) {
    const bool isx = i < ROWS;
    const int64_t c = isx ? static_cast<int64_t>(h) * kP + row0 + i
                          : hp + (i - ROWS < N ? static_cast<int64_t>(g) * N + (i - ROWS) : (p.ngroups + g) * N + (i - ROWS - N));
    const Row4 w = reinterpret_cast<const Row4 *>(p.w)[c];
    const int64_t rbase = ((slot < 0 ? 0 : slot) * channels + c) * p.ring_len;
    float v = p.wb ? p.wb[c] : 0.0f;
    const float now = load_io<IO>(p.xBC, b * p.xs + c);
    v = fmaf(w.v[kW - 1], now, v);
#pragma unroll
    for (int back = 1; back < kW; ++back)
      if (seen >= back) v = fmaf(w.v[kW - 1 - back], load_io<IO>(p.ring, rbase + static_cast<uint32_t>(seen - back) % p.ring_len), v);
    if (p.silu) v = silu_f(v);
    su[i] = v;
    if (slot >= 0 && (isx || (static_cast<uint32_t>(h) == g * p.per_group && row0 == 0))) {
      const int64_t at = rbase + static_cast<uint32_t>(seen) % p.ring_len, from = b * p.xs + c;   // the input as it is
      if constexpr (IO != 0) static_cast<uint16_t *>(p.ring)[at] = static_cast<const uint16_t *>(p.xBC)[from];
      else static_cast<uint32_t *>(p.ring)[at] = static_cast<const uint32_t *>(p.xBC)[from];
    }
  }
  float step = load_io<IO>(p.dt, b * p.dts + h) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
  if (p.softplus) step = softplus_step(step);
  if (p.dt_limit) step = fminf(fmaxf(step, p.dt_min), p.dt_max);
  const float keep = fast_exp2(step * p.A[h] * kLog2e);
  __syncthreads();

  // ---- state <- keep state + step x B, y = state C
  const f4 Bv = *reinterpret_cast<const f4 *>(&su[ROWS + n0]) * step, Cv = *reinterpret_cast<const f4 *>(&su[ROWS + N + n0]);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int row = r + i * AT_ONCE;
    if (row >= ROWS) break;
    const float xv = su[row];
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      st[i][k] = fmaf(keep, st[i][k], Bv[k] * xv);
      y = fmaf(Cv[k], st[i][k], y);
    }
    if (slot >= 0) __builtin_nontemporal_store(st[i], reinterpret_cast<f4 *>(srow + i * AT_ONCE * N));
    y = lane_sum<LPR>(y);
    if (tid % LPR == 0) {
      const int64_t ch = static_cast<int64_t>(h) * kP + row0 + row;
      if (p.D) y = fmaf(p.D_per_channel ? p.D[ch] : p.D[h], xv, y);
      if (p.z) y *= silu_f(load_io<IO>(p.z, b * p.zs + ch));
      store_one<IO>(p.out, b * p.os + ch, y);
    }
  }
}

template <int IO, int N>
void launch_step(int rows, dim3 grid, hipStream_t s, const StepParams &p) {
  if (rows == 64) hipLaunchKernelGGL((step_kernel<IO, N, 64>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((step_kernel<IO, N, 16>), grid, dim3(256), 0, s, p);
}
template <int IO>
void launch_step_n(int64_t n, int rows, dim3 grid, hipStream_t s, const StepParams &p) {
  if (n == 32) launch_step<IO, 32>(rows, grid, s, p);
  else if (n == 64) launch_step<IO, 64>(rows, grid, s, p);
  else launch_step<IO, 128>(rows, grid, s, p);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int conv1d_ssd_update(const conv1d_ssd_update_args_t *a, void *stream_ptr) {
  const int st = conv1d_ssd_update_validate(a);
  if (st != SSM_OK) return st;
  StepParams p{};
  p.xBC = a->xBC; p.xs = a->xBC_stride;
  p.dt = a->dt; p.dts = a->dt_stride;
  p.z = a->z; p.zs = a->z_stride;
  p.out = a->out; p.os = a->out_stride;
  p.A = a->A; p.w = a->conv_weight; p.wb = a->conv_bias; p.D = a->D; p.dt_bias = a->dt_bias;
  p.D_per_channel = a->D_per_channel;
  p.ring = a->conv_state; p.ring_len = static_cast<uint32_t>(a->state_len);
  p.state = a->ssm_state; p.nslots = a->state_slots;
  p.seen = a->cache_seqlens; p.slots = a->slots;
  p.nheads = a->nheads; p.ngroups = a->ngroups;
  p.per_group = static_cast<uint32_t>(a->nheads / a->ngroups);
  p.silu = a->act == SSM_ACT_SILU;
  p.softplus = a->dt_softplus;
  p.dt_limit = a->dt_limit; p.dt_min = a->dt_min; p.dt_max = a->dt_max;
  // Where the heads alone do not fill the chip four workgroups share one, each
  // of which forms B's and C's convolution again: 16 rows / 64 (us) of 256
  // (request, head) pairs 6.1 / 7.1 at dstate 128, 4.5 / 4.9 at 64, 3.9 / 3.8 at
  // 32, and of 512 10.9 / 8.5, 5.9 / 5.8, 4.8 / 4.3; of 32 4.4 / 6.2, of 1024
  // 17.5 / 12.8.
  const int rows = a->batch * a->nheads >= 2 * cu_count_cached() ? 64 : 16;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const dim3 grid(static_cast<unsigned>(a->nheads), kP / rows, static_cast<unsigned>(a->batch));
  if (a->io_dtype == SSM_BF16) launch_step_n<1>(a->dstate, rows, grid, stream, p);
  else if (a->io_dtype == SSM_F16) launch_step_n<2>(a->dstate, rows, grid, stream, p);
  else launch_step_n<0>(a->dstate, rows, grid, stream, p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}
