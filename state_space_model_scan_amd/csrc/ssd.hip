// ssd.hip -- the Mamba-2 chunked scan (ssd_scan_fwd) on the gfx950 matrix
// cores.
//
// Operation: the mamba2 chunk-scan operators the PaddleNLP Kernel
// operator-library guide lists in section 4.4 (mamba_chunk_scan_combined,
// chunk_state, state_passing), read as the selective-scan recurrence with a
// scalar decay per head; include/ssmscan.h writes it out.
//
// Evaluation (state-space duality).  Per (batch, head) and chunk of Q = 64
// tokens, with dt' the step, cs_t = A * sum_{k<=t} dt'_k inside the chunk
// and S the (headdim x dstate) state at the chunk's start:
//   M[t][tau]  = (C_t . B_tau) * exp(cs_t - cs_tau) * dt'_tau      (tau <= t)
//   Y          = M X + diag(exp(cs)) C S^T
//   S         <- exp(cs_last) S + X^T diag(exp(cs_last - cs) * dt') B
// which is the recurrence summed in another order.  The products run as
// v_mfma_f32_16x16x32_bf16 (bf16 operands, fp32 accumulation).  x, B and C
// are bf16 data and enter exactly; the three derived operands -- M, the
// state S in C S^T, and X scaled by the decay weights -- are split into a
// bf16 head and a bf16 tail (v = hi + lo, about 16 significant bits) and
// enter as two products each.  Rounding them to one bf16 instead costs 3-10%
// of the output (C S^T sums 128 terms with heavy cancellation); the split
// brings the error to about 1e-4.  The state stays in fp32 accumulators
// across chunks; C S^T takes its hi/lo split straight from them.
//
// Work decomposition: one 256-thread workgroup (four waves) per (batch,
// head), walking the chunks in order.  Wave w owns the chunk's tokens
// [16w, 16w+16) for M, and the head's channels [16w, 16w+16) for Y (all 64
// tokens) and for the state.  Operand layout of the 16x16x32 instruction
// (checked on the device): lane l holds A[l%16][8(l/16)+i] and
// B[8(l/16)+i][l%16] for i < 8, and accumulator i is D[4(l/16)+i][l%16].
// The products are taken transposed (G^T = B C^T, Y^T, S^T) so that each
// lane's four accumulators are consecutive elements of one LDS row and go
// out in one store; in C S^T the state operand is this lane's own
// accumulators, with the k index running over the states in their order
// and C read in the same order.  LDS matrices are row-major with each row's
// 16-byte groups (8-byte pieces for the C tile) permuted by the row index,
// so the operand reads and the transposed staging stores of X and B spread
// over the banks without padding (measured: bank conflicts were the largest
// stall before this layout).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_util.h"
#include "ssd_kernel.h"
#include "ssmscan.h"

namespace ssm {
namespace {

// state_passing: one thread per state element of a (batch, head), the chunks
// in order; S <- P S + E is one fp32 fma, as the fold in the full pass.
__global__ void __launch_bounds__(256) ssd_state_passing_kernel(const float *states, const float *decays,
                                                                const float *init, float *carried,
                                                                float *fin, int64_t nchunks, int64_t nbh,
                                                                int64_t ps) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= nbh * ps) return;
  const int64_t bh = i / ps;
  float S = init ? init[i] : 0.0f;
  for (int64_t c = 0; c < nchunks; ++c) {
    carried[c * nbh * ps + i] = S;
    S = fmaf(decays[c * nbh + bh], S, states[c * nbh * ps + i]);
  }
  if (fin) fin[i] = S;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct SsdPlan {
  int nseg;
  int64_t seg_chunks;
  size_t off_decay, ws_bytes;
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

using SsdFn = void (*)(const SsdParams);

template <int N>
SsdFn ssd_fn_n(int mode, bool seq) {
  if (mode == SSD_FULL) return seq ? ssd_kernel<N, SSD_FULL, true> : ssd_kernel<N, SSD_FULL, false>;
  return seq ? ssd_kernel<N, SSD_STATE, true> : ssd_kernel<N, SSD_STATE, false>;
}

SsdFn ssd_fn(int64_t dstate, int mode, bool seq) {
  switch (dstate) {
    case 32: return ssd_fn_n<32>(mode, seq);
    case 64: return ssd_fn_n<64>(mode, seq);
    default: return ssd_fn_n<128>(mode, seq);
  }
}

// Segments: a workgroup walks its (batch, head)'s chunks in order, so with
// few (batch, head) pairs the chunks are cut into G segments of whole
// chunks: enough workgroups for 1.5 times what the GPU holds at once, each
// segment at least two chunks.  More segments only add state-pass work:
// at b=8 l=2048 h=80 n=128 (640 pairs, 512 resident) one pass took 419 us,
// 2 segments 381, 3 392, 4 399, 8 464.
SsdPlan ssd_plan(const ssd_scan_args_t *a, int cus) {
  SsdPlan pl{};
  const int64_t nchunks = (a->seqlen + kQ - 1) / kQ;
  const int64_t BH = a->batch * a->nheads;
  int G = 1;
  if (a->seq_segments >= 1) {
    G = a->seq_segments;
  } else {
    int bf = blocks_per_cu(reinterpret_cast<const void *>(ssd_fn(a->dstate, SSD_FULL, a->seq_idx != nullptr)), 256);
    if (bf <= 0) bf = 2;
    const int64_t want = static_cast<int64_t>(bf) * cus * 3 / 2;
    if (BH < want) {
      int64_t g = (want + BH - 1) / BH;
      if (g > nchunks / 2) g = nchunks / 2;
      G = g > 1 ? static_cast<int>(g) : 1;
    }
  }
  if (G > nchunks) G = static_cast<int>(nchunks);
  pl.seg_chunks = (nchunks + G - 1) / G;
  pl.nseg = static_cast<int>((nchunks + pl.seg_chunks - 1) / pl.seg_chunks);
  // The library's own two-segment plan cuts the first segment short, about
  // 9/32 of the chunks, and the last segment takes the rest: the state pass
  // shrinks with the first segment, and the full pass, which starts the long
  // segment's workgroups first, fills the compute units with the short ones
  // (ssd2p7b, measured interleaved: first segment of 16 chunks 346 us, 8:
  // 326, 9: 319, 10: 324, 11: 331, 12: 341).
  if (a->seq_segments < 1 && pl.nseg == 2) {
    int64_t first = (9 * nchunks + 16) / 32;
    if (first < 2) first = 2;
    if (first < nchunks) pl.seg_chunks = first;
  }
  if (pl.nseg > 1) {
    const size_t ns = static_cast<size_t>(pl.nseg - 1) * BH;
    pl.off_decay = up256(ns * kP * a->dstate * sizeof(float));
    pl.ws_bytes = pl.off_decay + up256(ns * sizeof(float));
  }
  return pl;
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" int ssd_scan_workspace_size(const ssd_scan_args_t *a, size_t *bytes) {
  const int st = ssd_scan_validate(a);
  if (st != SSM_OK) return st;
  if (!bytes) return SSM_ERR_NULL;
  *bytes = ssd_plan(a, cu_count_cached()).ws_bytes;
  return SSM_OK;
}

namespace {

// the kernel parameters every launch shares
SsdParams ssd_params(const ssd_scan_args_t *a) {
  SsdParams p{};
  p.x = static_cast<const uint16_t *>(a->x);
  p.dt = static_cast<const uint16_t *>(a->dt);
  p.B = static_cast<const uint16_t *>(a->B);
  p.C = static_cast<const uint16_t *>(a->C);
  p.z = static_cast<const uint16_t *>(a->z);
  p.A = a->A; p.D = a->D; p.dt_bias = a->dt_bias; p.init = a->initial_states;
  p.seq_idx = a->seq_idx;
  p.out = static_cast<uint16_t *>(a->out);
  p.fin = a->final_states;
  p.seqlen = a->seqlen; p.nheads = a->nheads; p.ngroups = a->ngroups;
  p.D_per_channel = a->D_per_channel;
  p.softplus = a->dt_softplus;
  p.dt_limit = a->dt_limit; p.dt_min = a->dt_min; p.dt_max = a->dt_max;
  return p;
}

}  // namespace

extern "C" int ssd_chunk_state(const ssd_scan_args_t *a, int64_t chunk_size, float *states, float *decays,
                               void *stream_ptr) {
  const int st = ssd_chunk_state_validate(a, chunk_size, states, decays);
  if (st != SSM_OK) return st;
  const int64_t nchunks = (a->seqlen + chunk_size - 1) / chunk_size;
  const int64_t blocks = a->batch * a->nheads;
  if (blocks > 0x7fffffffLL || nchunks > 65535) return SSM_ERR_SHAPE;
  SsdParams p = ssd_params(a);
  p.C = nullptr; p.z = nullptr; p.D = nullptr; p.init = nullptr; p.out = nullptr; p.fin = nullptr;
  p.nseg = static_cast<int>(nchunks);
  p.seg_chunks = chunk_size / kQ;
  p.ws_state = states;
  p.ws_decay = decays;
  hipLaunchKernelGGL(ssd_fn(a->dstate, SSD_STATE, a->seq_idx != nullptr),
                     dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(nchunks)), dim3(256), 0,
                     static_cast<hipStream_t>(stream_ptr), p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

extern "C" int ssd_state_passing(int64_t nchunks, int64_t batch, int64_t nheads, int64_t headdim,
                                 int64_t dstate, const float *states, const float *decays,
                                 const float *initial_states, float *carried, float *final_states,
                                 void *stream_ptr) {
  const int st = ssd_state_passing_validate(nchunks, batch, nheads, headdim, dstate, states, decays, carried);
  if (st != SSM_OK) return st;
  const int64_t nbh = batch * nheads, ps = headdim * dstate;
  const int64_t blocks = (nbh * ps + 255) / 256;
  if (blocks > 0x7fffffffLL) return SSM_ERR_SHAPE;
  hipLaunchKernelGGL(ssd_state_passing_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                     static_cast<hipStream_t>(stream_ptr), states, decays, initial_states, carried,
                     final_states, nchunks, nbh, ps);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

extern "C" int ssd_chunk_scan(const ssd_scan_args_t *a, int64_t chunk_size, const float *carried,
                              void *stream_ptr) {
  const int st = ssd_chunk_scan_validate(a, chunk_size, carried);
  if (st != SSM_OK) return st;
  const int64_t nchunks = (a->seqlen + chunk_size - 1) / chunk_size;
  const int64_t blocks = a->batch * a->nheads;
  if (blocks > 0x7fffffffLL || nchunks > 65535) return SSM_ERR_SHAPE;
  SsdParams p = ssd_params(a);
  p.init = nullptr;
  p.carried = carried;
  p.nseg = static_cast<int>(nchunks);
  p.seg_chunks = chunk_size / kQ;
  hipLaunchKernelGGL(ssd_fn(a->dstate, SSD_FULL, a->seq_idx != nullptr),
                     dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(nchunks)), dim3(256), 0,
                     static_cast<hipStream_t>(stream_ptr), p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SSM_OK : hip_fail(e);
}

extern "C" int ssd_scan_fwd(const ssd_scan_args_t *a, void *stream_ptr) {
  const int st = ssd_scan_validate(a);
  if (st != SSM_OK) return st;
  const SsdPlan pl = ssd_plan(a, cu_count_cached());
  if (pl.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < pl.ws_bytes)) return SSM_ERR_WORKSPACE;
  SsdParams p = ssd_params(a);
  p.nseg = pl.nseg; p.seg_chunks = pl.seg_chunks;
  if (pl.nseg > 1) {
    char *ws = static_cast<char *>(a->workspace);
    p.ws_state = reinterpret_cast<float *>(ws);
    p.ws_decay = reinterpret_cast<float *>(ws + pl.off_decay);
  }
  const int64_t blocks = a->batch * a->nheads;
  if (blocks > 0x7fffffffLL) return SSM_ERR_SHAPE;
  hipStream_t stream = static_cast<hipStream_t>(stream_ptr);
  const unsigned gx = static_cast<unsigned>(blocks);
  const bool seq = a->seq_idx != nullptr;
  if (pl.nseg > 1) {
    hipLaunchKernelGGL(ssd_fn(a->dstate, SSD_STATE, seq), dim3(gx, pl.nseg - 1), dim3(256), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_fail(e);
  }
  hipLaunchKernelGGL(ssd_fn(a->dstate, SSD_FULL, seq), dim3(gx, pl.nseg), dim3(256), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e);
  return SSM_OK;
}
