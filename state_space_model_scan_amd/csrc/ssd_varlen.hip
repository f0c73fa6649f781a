// ssd_varlen.hip -- the Mamba-2 chunked scan over packed tokens
// (ssd_varlen_fwd): prompts of several lengths from and to a cache of states,
// and the training forward, which keeps every chunk's entering state in 8
// bits.  The kernel is ssd_kernel.h's with VAR set.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_util.h"
#include "ssd_kernel.h"
#include "ssmscan.h"

namespace ssm {
namespace {

using VarFn = void (*)(const SsdParams);

VarFn var_fn(int64_t dstate, int mode) {
  const bool full = mode == SSD_FULL;
  switch (dstate) {
    case 32: return full ? ssd_kernel<32, SSD_FULL, false, true> : ssd_kernel<32, SSD_STATE, false, true>;
    case 64: return full ? ssd_kernel<64, SSD_FULL, false, true> : ssd_kernel<64, SSD_STATE, false, true>;
    default: return full ? ssd_kernel<128, SSD_FULL, false, true> : ssd_kernel<128, SSD_STATE, false, true>;
  }
}

struct VarPlan {
  int nseg;
  int64_t seg_chunks;
  size_t off_decay, ws_bytes;
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Segments of the longest sequence; a shorter one has fewer.  Enough
// workgroups for 1.5 times what the GPU holds at once, each segment at least
// two chunks, as for dense rows.
VarPlan var_plan(const ssd_varlen_args_t *a, int cus) {
  VarPlan pl{};
  int64_t nchunks = (a->max_seqlen + kQ - 1) / kQ;
  if (nchunks < 1) nchunks = 1;
  const int64_t SH = a->nseq * a->nheads;
  int64_t G = 1;
  if (a->seq_segments >= 1) {
    G = a->seq_segments;
  } else {
    int per_cu = blocks_per_cu(reinterpret_cast<const void *>(var_fn(a->dstate, SSD_FULL)), 256);
    if (per_cu <= 0) per_cu = 2;
    // workgroups that have tokens: ragged sequences fill a part of the grid
    const int64_t chunks = a->total / kQ + a->nseq;
    const int64_t full_rows = (chunks + nchunks - 1) / nchunks;
    const int64_t busy = (full_rows < a->nseq ? full_rows : a->nseq) * a->nheads;
    const int64_t want = static_cast<int64_t>(per_cu) * cus * 3 / 2;
    if (busy < want) G = (want + busy - 1) / busy;
    if (G > nchunks / 2) G = nchunks / 2;
    if (G < 1) G = 1;
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
  const int64_t blocks = a->nseq * a->nheads;
  if (blocks > 0x7fffffffLL) return SSM_ERR_SHAPE;
  SsdParams p{};
  p.x = static_cast<const uint16_t *>(a->x); p.xs = a->x_stride;
  p.dt = static_cast<const uint16_t *>(a->dt); p.dts = a->dt_stride;
  p.B = static_cast<const uint16_t *>(a->B); p.bs = a->B_stride;
  p.C = static_cast<const uint16_t *>(a->C); p.cs = a->C_stride;
  p.z = static_cast<const uint16_t *>(a->z); p.zs = a->z_stride;
  p.out = static_cast<uint16_t *>(a->out); p.os = a->out_stride;
  p.A = a->A; p.D = a->D; p.dt_bias = a->dt_bias;
  p.D_per_channel = a->D_per_channel;
  p.softplus = a->dt_softplus;
  p.dt_limit = a->dt_limit; p.dt_min = a->dt_min; p.dt_max = a->dt_max;
  p.nheads = a->nheads; p.ngroups = a->ngroups;
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
    hipLaunchKernelGGL(var_fn(a->dstate, SSD_STATE), dim3(gx, pl.nseg - 1), dim3(256), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_fail(e);
  }
  hipLaunchKernelGGL(var_fn(a->dstate, SSD_FULL), dim3(gx, pl.nseg), dim3(256), 0, stream, p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}
