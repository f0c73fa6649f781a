// Host-side argument checks of the C ABI.  Plain C++: no HIP header, no device
// access, so every error path can be exercised on a machine without a GPU.
//
// What is checked follows the argument list of selective_scan_fn and
// causal_conv1d_fn (PaddleNLP Kernel operator-library guide, sections 4.1 and
// 4.2): required tensors present, positive sizes, dim divisible by the number
// of B/C groups, one of the supported io dtypes, dstate within the compiled
// range, and the conv width and activation the kernels are built for.
#include "ssmscan.h"

#include <cstdint>
#include <limits>

namespace {

bool positive(int64_t v) { return v > 0; }

// b*d*l (and friends) must fit comfortably in int64 element counts.
bool product_fits(int64_t a, int64_t b, int64_t c) {
  const int64_t lim = std::numeric_limits<int64_t>::max() / 8;
  if (a > lim / b) return false;
  const int64_t ab = a * b;
  return ab <= lim / c;
}

}  // namespace

extern "C" int ssm_scan_validate(const ssm_scan_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->batch) || !positive(a->dim) || !positive(a->seqlen) ||
      !positive(a->dstate) || !positive(a->ngroups))
    return SSM_ERR_SHAPE;
  if (a->dim % a->ngroups != 0) return SSM_ERR_SHAPE;
  if (a->seq_segments < 0) return SSM_ERR_SHAPE;
  if (!product_fits(a->batch, a->dim, a->seqlen) ||
      !product_fits(a->batch, a->ngroups * a->dstate, a->seqlen))
    return SSM_ERR_SHAPE;
  if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16 && a->io_dtype != SSM_F16) return SSM_ERR_UNSUPPORTED;
  if (a->dstate > SSM_MAX_DSTATE) return SSM_ERR_UNSUPPORTED;
  if ((a->B_kind != SSM_BC_FIXED && a->B_kind != SSM_BC_VARYING) ||
      (a->C_kind != SSM_BC_FIXED && a->C_kind != SSM_BC_VARYING))
    return SSM_ERR_UNSUPPORTED;
  if (a->delta_softplus != 0 && a->delta_softplus != 1) return SSM_ERR_UNSUPPORTED;
  if (!a->delta || !a->A || !a->B || !a->C || !a->out) return SSM_ERR_NULL;
  if (a->conv_weight) {
    if (!a->conv_x) return SSM_ERR_NULL;
    if (a->conv_width != SSM_CONV_WIDTH) return SSM_ERR_UNSUPPORTED;
    if (a->conv_act != SSM_ACT_NONE && a->conv_act != SSM_ACT_SILU) return SSM_ERR_UNSUPPORTED;
  } else if (!a->u) {
    return SSM_ERR_NULL;
  }
  return SSM_OK;
}

// selective_scan_fn with complex A (guide section 4.1): the checks of the
// real scan, with B/C holding (real, imaginary) pairs; no conv prologue and
// no checkpoints.
extern "C" int ssm_scan_complex_validate(const ssm_scan_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  const int st = ssm_scan_validate(a);
  if (st != SSM_OK) return st;
  if (!product_fits(a->batch, 2 * a->ngroups * a->dstate, a->seqlen)) return SSM_ERR_SHAPE;
  if (a->conv_weight) return SSM_ERR_UNSUPPORTED;
  if (!a->u) return SSM_ERR_NULL;
  return SSM_OK;
}

extern "C" int causal_conv1d_ex_validate(const causal_conv1d_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  const int st = causal_conv1d_validate(a->x, a->weight, a->out, a->batch, a->dim, a->seqlen, a->width,
                                        a->io_dtype, a->act);
  if (st != SSM_OK) return st;
  // the page: seq_idx excludes initial_states and the final states
  if (a->seq_idx && (a->initial_states || a->final_states)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

extern "C" int ssm_scan_bwd_validate(const ssm_scan_bwd_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->batch) || !positive(a->dim) || !positive(a->seqlen) ||
      !positive(a->dstate) || !positive(a->ngroups))
    return SSM_ERR_SHAPE;
  if (a->dim % a->ngroups != 0) return SSM_ERR_SHAPE;
  // the per-workgroup partial sums hold up to (batch*ngroups, dim, dstate, seqlen) floats
  if (!product_fits(a->batch, a->dim, a->seqlen) ||
      !product_fits(a->batch * a->dim, a->dstate, a->seqlen))
    return SSM_ERR_SHAPE;
  if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16 && a->io_dtype != SSM_F16) return SSM_ERR_UNSUPPORTED;
  if (a->dstate > SSM_MAX_DSTATE) return SSM_ERR_UNSUPPORTED;
  if ((a->B_kind != SSM_BC_FIXED && a->B_kind != SSM_BC_VARYING) ||
      (a->C_kind != SSM_BC_FIXED && a->C_kind != SSM_BC_VARYING))
    return SSM_ERR_UNSUPPORTED;
  if (a->delta_softplus != 0 && a->delta_softplus != 1) return SSM_ERR_UNSUPPORTED;
  if (a->seq_segments < 0) return SSM_ERR_SHAPE;
  if (!a->u || !a->delta || !a->A || !a->B || !a->C || !a->checkpoints || !a->dout ||
      !a->du || !a->ddelta || !a->dA || !a->dB || !a->dC)
    return SSM_ERR_NULL;
  if ((a->z && !a->dz) || (a->D && !a->dD) || (a->delta_bias && !a->ddelta_bias)) return SSM_ERR_NULL;
  return SSM_OK;
}

extern "C" int ssm_scan_bwd_complex_validate(const ssm_scan_bwd_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  const int st = ssm_scan_bwd_validate(a);
  if (st != SSM_OK) return st;
  // complex B/C are pairs: twice the elements of the real layout
  if (!product_fits(a->batch, 2 * a->ngroups * a->dstate, a->seqlen) ||
      !product_fits(a->batch * a->dim, 2 * a->dstate, a->seqlen))
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

extern "C" int causal_conv1d_validate(const void *x, const float *weight, const void *out,
                                      int64_t batch, int64_t dim, int64_t seqlen,
                                      int32_t width, int32_t io_dtype, int32_t act) {
  if (!positive(batch) || !positive(dim) || !positive(seqlen)) return SSM_ERR_SHAPE;
  if (!product_fits(batch, dim, seqlen)) return SSM_ERR_SHAPE;
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16 && io_dtype != SSM_F16) return SSM_ERR_UNSUPPORTED;
  if (width != SSM_CONV_WIDTH) return SSM_ERR_UNSUPPORTED;
  if (act != SSM_ACT_NONE && act != SSM_ACT_SILU) return SSM_ERR_UNSUPPORTED;
  if (!x || !weight || !out) return SSM_ERR_NULL;
  return SSM_OK;
}

// selective_state_update (guide section 4.4 operator list) and
// causal_conv1d_update (section 4.2): the decode forms of the two operators.
extern "C" int ssm_state_update_validate(const ssm_state_update_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->batch) || !positive(a->dim) || !positive(a->dstate) || !positive(a->ngroups))
    return SSM_ERR_SHAPE;
  if (a->dim % a->ngroups != 0) return SSM_ERR_SHAPE;
  if (!product_fits(a->batch, a->dim, a->dstate) || !product_fits(a->batch, a->ngroups, a->dstate))
    return SSM_ERR_SHAPE;
  if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16 && a->io_dtype != SSM_F16) return SSM_ERR_UNSUPPORTED;
  if (a->dstate > SSM_MAX_DSTATE) return SSM_ERR_UNSUPPORTED;
  if (a->dt_softplus != 0 && a->dt_softplus != 1) return SSM_ERR_UNSUPPORTED;
  if (!a->state || !a->x || !a->dt || !a->A || !a->B || !a->C || !a->out) return SSM_ERR_NULL;
  return SSM_OK;
}

extern "C" int causal_conv1d_update_validate(const void *x, const void *conv_state,
                                             const float *weight, const void *out,
                                             int64_t batch, int64_t dim, int64_t seqlen,
                                             int64_t state_len, int32_t width,
                                             int32_t io_dtype, int32_t act) {
  if (!positive(batch) || !positive(dim) || !positive(seqlen) || !positive(state_len))
    return SSM_ERR_SHAPE;
  if (!product_fits(batch, dim, seqlen) || !product_fits(batch, dim, state_len)) return SSM_ERR_SHAPE;
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16 && io_dtype != SSM_F16) return SSM_ERR_UNSUPPORTED;
  if (width < 2 || width > SSM_CONV_WIDTH) return SSM_ERR_UNSUPPORTED;
  if (state_len < width - 1) return SSM_ERR_SHAPE;
  if (state_len > SSM_MAX_CONV_STATE) return SSM_ERR_UNSUPPORTED;
  if (act != SSM_ACT_NONE && act != SSM_ACT_SILU) return SSM_ERR_UNSUPPORTED;
  if (!x || !conv_state || !weight || !out) return SSM_ERR_NULL;
  return SSM_OK;
}

// Mamba-2 chunked scan (guide section 4.4 operator list).
extern "C" int ssd_scan_validate(const ssd_scan_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->batch) || !positive(a->seqlen) || !positive(a->nheads) ||
      !positive(a->headdim) || !positive(a->dstate) || !positive(a->ngroups))
    return SSM_ERR_SHAPE;
  if (a->nheads % a->ngroups != 0) return SSM_ERR_SHAPE;
  if (!product_fits(a->batch * a->seqlen, a->nheads, a->headdim) ||
      !product_fits(a->batch * a->seqlen, a->ngroups, a->dstate) ||
      !product_fits(a->batch, a->nheads, a->headdim * a->dstate))
    return SSM_ERR_SHAPE;
  if (a->io_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (a->headdim != SSD_HEADDIM) return SSM_ERR_UNSUPPORTED;
  if (a->dstate != 32 && a->dstate != 64 && a->dstate != 128) return SSM_ERR_UNSUPPORTED;
  if (a->dt_softplus != 0 && a->dt_softplus != 1) return SSM_ERR_UNSUPPORTED;
  if (a->D_per_channel != 0 && a->D_per_channel != 1) return SSM_ERR_UNSUPPORTED;
  if (a->dt_limit != 0 && a->dt_limit != 1) return SSM_ERR_UNSUPPORTED;
  if (a->dt_limit && !(a->dt_min <= a->dt_max)) return SSM_ERR_SHAPE;
  if (a->seq_segments < 0) return SSM_ERR_SHAPE;
  if (!a->x || !a->dt || !a->A || !a->B || !a->C || !a->out) return SSM_ERR_NULL;
  const uintptr_t mis = (reinterpret_cast<uintptr_t>(a->x) | reinterpret_cast<uintptr_t>(a->B) |
                         reinterpret_cast<uintptr_t>(a->C) | reinterpret_cast<uintptr_t>(a->out) |
                         reinterpret_cast<uintptr_t>(a->z)) & 15u;
  if (mis) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// the checks of ssd_scan_validate that the split operators share: sizes,
// dtypes, enum values, and x / dt / A / B present and aligned
static int ssd_common_validate(const ssd_scan_args_t *a, int64_t chunk_size) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->batch) || !positive(a->seqlen) || !positive(a->nheads) ||
      !positive(a->headdim) || !positive(a->dstate) || !positive(a->ngroups))
    return SSM_ERR_SHAPE;
  if (a->nheads % a->ngroups != 0) return SSM_ERR_SHAPE;
  if (!product_fits(a->batch * a->seqlen, a->nheads, a->headdim) ||
      !product_fits(a->batch * a->seqlen, a->ngroups, a->dstate) ||
      !product_fits(a->batch, a->nheads, a->headdim * a->dstate))
    return SSM_ERR_SHAPE;
  if (a->io_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (a->headdim != SSD_HEADDIM) return SSM_ERR_UNSUPPORTED;
  if (a->dstate != 32 && a->dstate != 64 && a->dstate != 128) return SSM_ERR_UNSUPPORTED;
  if (a->dt_softplus != 0 && a->dt_softplus != 1) return SSM_ERR_UNSUPPORTED;
  if (a->dt_limit != 0 && a->dt_limit != 1) return SSM_ERR_UNSUPPORTED;
  if (a->dt_limit && !(a->dt_min <= a->dt_max)) return SSM_ERR_SHAPE;
  if (chunk_size <= 0 || chunk_size % SSD_CHUNK != 0) return SSM_ERR_UNSUPPORTED;
  if (!a->x || !a->dt || !a->A || !a->B) return SSM_ERR_NULL;
  const int64_t nchunks = (a->seqlen + chunk_size - 1) / chunk_size;
  if (!product_fits(nchunks, a->batch * a->nheads, a->headdim * a->dstate)) return SSM_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(a->x) | reinterpret_cast<uintptr_t>(a->B)) & 15u) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

extern "C" int ssd_chunk_state_validate(const ssd_scan_args_t *a, int64_t chunk_size, const float *states,
                                        const float *decays) {
  const int st = ssd_common_validate(a, chunk_size);
  if (st != SSM_OK) return st;
  if (!states || !decays) return SSM_ERR_NULL;
  return SSM_OK;
}

extern "C" int ssd_chunk_scan_validate(const ssd_scan_args_t *a, int64_t chunk_size, const float *carried) {
  const int st = ssd_common_validate(a, chunk_size);
  if (st != SSM_OK) return st;
  if (a->D_per_channel != 0 && a->D_per_channel != 1) return SSM_ERR_UNSUPPORTED;
  if (!a->C || !a->out || !carried) return SSM_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(a->C) | reinterpret_cast<uintptr_t>(a->out) |
       reinterpret_cast<uintptr_t>(a->z)) & 15u)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

extern "C" int ssd_state_passing_validate(int64_t nchunks, int64_t batch, int64_t nheads, int64_t headdim,
                                          int64_t dstate, const float *states, const float *decays,
                                          const float *carried) {
  if (!positive(nchunks) || !positive(batch) || !positive(nheads) || !positive(headdim) || !positive(dstate))
    return SSM_ERR_SHAPE;
  if (!product_fits(nchunks, batch * nheads, headdim * dstate) || !product_fits(batch, nheads, headdim * dstate))
    return SSM_ERR_SHAPE;
  if (!states || !decays || !carried) return SSM_ERR_NULL;
  return SSM_OK;
}

// Packed tokens: the short conv, the chunked scan and its step.
namespace {

bool io_ok(int32_t io) { return io == SSM_F32 || io == SSM_BF16 || io == SSM_F16; }
bool flag_ok(int32_t v) { return v == 0 || v == 1; }
uintptr_t bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

int conv_varlen_common(const causal_conv1d_varlen_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->total) || !positive(a->nseq) || !positive(a->channels)) return SSM_ERR_SHAPE;
  if (a->total > 0x7fffffffLL || a->nseq > 0x7fffffffLL) return SSM_ERR_SHAPE;   // int32 edges
  if (a->channels > 0x7fffffffLL || a->x_stride < a->channels || !product_fits(a->total, a->x_stride, 1))
    return SSM_ERR_SHAPE;
  if (!io_ok(a->io_dtype)) return SSM_ERR_UNSUPPORTED;
  if (a->width != SSM_CONV_WIDTH) return SSM_ERR_UNSUPPORTED;
  if (a->act != SSM_ACT_NONE && a->act != SSM_ACT_SILU) return SSM_ERR_UNSUPPORTED;
  if (!a->x || !a->weight || !a->cu_seqlens) return SSM_ERR_NULL;
  return SSM_OK;
}

// what the packed scan's forward and backward share
// The longest stride with which a chunk's tokens are reached by 32-bit byte offsets.
constexpr int64_t kFarRow = (int64_t{1} << 31) / (2 * SSD_CHUNK);

int ssd_varlen_common(const ssd_varlen_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->total) || !positive(a->nseq) || a->max_seqlen < 0 || !positive(a->nheads) ||
      !positive(a->headdim) || !positive(a->dstate) || !positive(a->ngroups))
    return SSM_ERR_SHAPE;
  if (a->total > 0x7fffffffLL || a->nseq > 0x7fffffffLL || a->max_seqlen > a->total) return SSM_ERR_SHAPE;
  if (a->nheads > 65535 || a->nheads % a->ngroups != 0) return SSM_ERR_SHAPE;
  if (a->io_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (a->headdim != SSD_HEADDIM) return SSM_ERR_UNSUPPORTED;
  if (a->dstate != 32 && a->dstate != 64 && a->dstate != 128) return SSM_ERR_UNSUPPORTED;
  const int64_t hp = a->nheads * a->headdim, gn = a->ngroups * a->dstate;
  if (a->x_stride < hp || a->B_stride < gn || a->C_stride < gn || a->dt_stride < a->nheads ||
      !product_fits(a->total, a->x_stride, 1) || !product_fits(a->total, a->B_stride, 1) ||
      !product_fits(a->total, a->C_stride, 1) || !product_fits(a->total, a->dt_stride, 1) ||
      !product_fits(a->total / SSD_CHUNK + a->nseq, hp, a->dstate))
    return SSM_ERR_SHAPE;
  if (a->x_stride > kFarRow || a->B_stride > kFarRow || a->C_stride > kFarRow) return SSM_ERR_SHAPE;
  if (!flag_ok(a->D_per_channel) || !flag_ok(a->dt_softplus) || !flag_ok(a->dt_limit)) return SSM_ERR_UNSUPPORTED;
  if (a->dt_limit && !(a->dt_min <= a->dt_max)) return SSM_ERR_SHAPE;
  if (a->seq_segments < 0) return SSM_ERR_SHAPE;
  if (!a->x || !a->dt || !a->A || !a->B || !a->C || !a->cu_seqlens) return SSM_ERR_NULL;
  if ((bits(a->x) | bits(a->B) | bits(a->C)) & 15u) return SSM_ERR_UNSUPPORTED;
  if ((a->x_stride | a->B_stride | a->C_stride) & 7) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

}  // namespace

extern "C" int causal_conv1d_varlen_fwd_validate(const causal_conv1d_varlen_args_t *a) {
  const int st = conv_varlen_common(a);
  if (st != SSM_OK) return st;
  if (!a->out) return SSM_ERR_NULL;
  if (a->out_stride < a->channels || !product_fits(a->total, a->out_stride, 1)) return SSM_ERR_SHAPE;
  if (a->conv_state) {
    if (!positive(a->state_slots) || a->state_len < a->width) return SSM_ERR_SHAPE;
    if (a->state_len > SSM_MAX_CONV_STATE) return SSM_ERR_UNSUPPORTED;
    if (!product_fits(a->state_slots, a->channels, a->state_len)) return SSM_ERR_SHAPE;
  }
  return SSM_OK;
}

extern "C" int causal_conv1d_varlen_bwd_validate(const causal_conv1d_varlen_args_t *a) {
  const int st = conv_varlen_common(a);
  if (st != SSM_OK) return st;
  if (!a->dout || !a->dx || !a->dweight || (a->bias && !a->dbias)) return SSM_ERR_NULL;
  if (a->dout_stride < a->channels || a->dx_stride < a->channels || !product_fits(a->total, a->dout_stride, 1) ||
      !product_fits(a->total, a->dx_stride, 1))
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

extern "C" int64_t ssd_checkpoint_slots(int64_t total, int64_t nseq) { return total / SSD_CHUNK + nseq; }

extern "C" int ssd_varlen_fwd_validate(const ssd_varlen_args_t *a) {
  const int st = ssd_varlen_common(a);
  if (st != SSM_OK) return st;
  if (!a->out || (!a->checkpoints) != (!a->checkpoint_scales)) return SSM_ERR_NULL;
  const int64_t hp = a->nheads * a->headdim;
  if (a->out_stride < hp || !product_fits(a->total, a->out_stride, 1)) return SSM_ERR_SHAPE;
  if ((bits(a->out) & 15u) || (a->out_stride & 7)) return SSM_ERR_UNSUPPORTED;
  if (a->z) {
    if (a->z_stride < hp || !product_fits(a->total, a->z_stride, 1)) return SSM_ERR_SHAPE;
    if ((bits(a->z) & 15u) || (a->z_stride & 7)) return SSM_ERR_UNSUPPORTED;
  }
  if (a->ssm_state && (!positive(a->state_slots) || !product_fits(a->state_slots, hp, a->dstate))) return SSM_ERR_SHAPE;
  if (bits(a->ssm_state) & 15u || bits(a->checkpoints) & 15u) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

extern "C" int ssd_varlen_bwd_validate(const ssd_varlen_bwd_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  const ssd_varlen_args_t &f = a->fwd;
  const int st = ssd_varlen_common(&f);
  if (st != SSM_OK) return st;
  if (f.z) return SSM_ERR_UNSUPPORTED;
  if (!f.checkpoints || !f.checkpoint_scales || !a->dout || !a->dx || !a->ddt || !a->dB || !a->dC || !a->dA ||
      (f.D && !a->dD) || (f.dt_bias && !a->ddt_bias))
    return SSM_ERR_NULL;
  const int64_t hp = f.nheads * f.headdim, gn = f.ngroups * f.dstate, pn = f.headdim * f.dstate;
  const int64_t entries = ssd_checkpoint_slots(f.total, f.nseq);
  if ((entries > 1 && (a->code_entry_stride < pn || a->scale_entry_stride < f.headdim)) ||
      (f.nheads > 1 && (a->code_head_stride < pn || a->scale_head_stride < f.headdim)))
    return SSM_ERR_SHAPE;
  if (!product_fits(entries, a->code_entry_stride > 0 ? a->code_entry_stride : 1, 1) ||
      !product_fits(f.nheads, a->code_head_stride > 0 ? a->code_head_stride : 1, 1) ||
      !product_fits(entries, a->scale_entry_stride > 0 ? a->scale_entry_stride : 1, 1) ||
      !product_fits(f.nheads, a->scale_head_stride > 0 ? a->scale_head_stride : 1, 1))
    return SSM_ERR_SHAPE;
  if ((a->code_entry_stride | a->code_head_stride) & 15) return SSM_ERR_UNSUPPORTED;
  if (a->dout_stride > kFarRow) return SSM_ERR_SHAPE;
  if (a->dout_stride < hp || a->dx_stride < hp || a->ddt_stride < f.nheads || a->dB_stride < gn || a->dC_stride < gn ||
      !product_fits(f.total, a->dout_stride, 1) || !product_fits(f.total, a->dx_stride, 1) ||
      !product_fits(f.total, a->ddt_stride, 1) || !product_fits(f.total, a->dB_stride, 1) ||
      !product_fits(f.total, a->dC_stride, 1))
    return SSM_ERR_SHAPE;
  if ((bits(a->dout) | bits(a->dx) | bits(a->dB) | bits(a->dC) | bits(f.checkpoints) | bits(a->dfinal_states) |
       bits(a->dinitial_states)) & 15u)
    return SSM_ERR_UNSUPPORTED;
  if ((a->dout_stride | a->dx_stride | a->dB_stride | a->dC_stride) & 7) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

extern "C" int conv1d_ssd_update_validate(const conv1d_ssd_update_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->batch) || !positive(a->nheads) || !positive(a->headdim) || !positive(a->dstate) ||
      !positive(a->ngroups) || !positive(a->state_slots))
    return SSM_ERR_SHAPE;
  if (a->batch > 65535 || a->nheads > 65535 || a->nheads % a->ngroups != 0) return SSM_ERR_SHAPE;   // the grid
  if (!io_ok(a->io_dtype) || a->headdim != SSD_HEADDIM) return SSM_ERR_UNSUPPORTED;
  if (a->dstate != 32 && a->dstate != 64 && a->dstate != 128) return SSM_ERR_UNSUPPORTED;
  if (a->width != SSM_CONV_WIDTH || a->state_len > SSM_MAX_CONV_STATE) return SSM_ERR_UNSUPPORTED;
  if (a->act != SSM_ACT_NONE && a->act != SSM_ACT_SILU) return SSM_ERR_UNSUPPORTED;
  if (!flag_ok(a->D_per_channel) || !flag_ok(a->dt_softplus) || !flag_ok(a->dt_limit)) return SSM_ERR_UNSUPPORTED;
  if (a->dt_limit && !(a->dt_min <= a->dt_max)) return SSM_ERR_SHAPE;
  const int64_t hp = a->nheads * a->headdim, c = hp + 2 * a->ngroups * a->dstate;
  if (a->state_len < a->width || a->xBC_stride < c || a->dt_stride < a->nheads || a->out_stride < hp ||
      (a->z && a->z_stride < hp))
    return SSM_ERR_SHAPE;
  if (!product_fits(a->batch, a->xBC_stride, 1) || !product_fits(a->batch, a->dt_stride, 1) ||
      !product_fits(a->batch, a->out_stride, 1) || (a->z && !product_fits(a->batch, a->z_stride, 1)) ||
      !product_fits(a->state_slots, hp, a->dstate) || !product_fits(a->state_slots, c, a->state_len))
    return SSM_ERR_SHAPE;
  if (!a->xBC || !a->dt || !a->A || !a->conv_weight || !a->conv_state || !a->ssm_state || !a->out) return SSM_ERR_NULL;
  if (bits(a->ssm_state) & 15u) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// A gated recurrent block: its recurrence over packed tokens, and its norm.
namespace {

bool rows_fit(int64_t rows, int64_t cols, int64_t stride) { return stride >= cols && product_fits(rows, stride, 1); }
// ... and a wave's 16 tokens are reached by 32-bit offsets.
bool near_rows(int64_t rows, int64_t cols, int64_t stride) { return rows_fit(rows, cols, stride) && stride <= kFarRow; }

int gated_common(const gated_scan_varlen_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->total) || !positive(a->nseq) || !positive(a->channels)) return SSM_ERR_SHAPE;
  if (a->total > 0x7fffffffLL || a->nseq > 0x7fffffffLL || a->channels > 0x7fffffffLL) return SSM_ERR_SHAPE;   // int32 edges
  if (!near_rows(a->total, a->channels, a->x_stride) || !near_rows(a->total, a->channels, a->r_stride) ||
      !near_rows(a->total, a->channels, a->i_stride) || !product_fits(a->nseq, a->channels, 1))
    return SSM_ERR_SHAPE;
  if (!io_ok(a->io_dtype)) return SSM_ERR_UNSUPPORTED;
  if (!a->x || !a->r || !a->i || !a->A || !a->cu_seqlens) return SSM_ERR_NULL;
  return SSM_OK;
}

}  // namespace

extern "C" int64_t gated_checkpoint_slots(int64_t total) { return total / GATED_CHUNK + (total % GATED_CHUNK > 0); }

extern "C" int gated_scan_varlen_fwd_validate(const gated_scan_varlen_args_t *a) {
  const int st = gated_common(a);
  if (st != SSM_OK) return st;
  if (!a->out) return SSM_ERR_NULL;
  if (!near_rows(a->total, a->channels, a->out_stride)) return SSM_ERR_SHAPE;
  if (a->state && (!positive(a->state_slots) || !product_fits(a->state_slots, a->channels, 1))) return SSM_ERR_SHAPE;
  return SSM_OK;
}

extern "C" int gated_scan_varlen_bwd_validate(const gated_scan_varlen_bwd_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  const gated_scan_varlen_args_t &f = a->fwd;
  const int st = gated_common(&f);
  if (st != SSM_OK) return st;
  if (!f.checkpoints || !a->dout || !a->dx || !a->dr || !a->di || !a->dA || (f.r_bias && !a->dr_bias) ||
      (f.i_bias && !a->di_bias))
    return SSM_ERR_NULL;
  if (!near_rows(f.total, f.channels, a->dout_stride) || !near_rows(f.total, f.channels, a->dx_stride) ||
      !near_rows(f.total, f.channels, a->dr_stride) || !near_rows(f.total, f.channels, a->di_stride))
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

extern "C" int gated_scan_update_validate(const gated_scan_update_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  if (!positive(a->batch) || !positive(a->channels) || !positive(a->state_slots)) return SSM_ERR_SHAPE;
  if (a->batch > 0x7fffffffLL || a->channels > 0x7fffffffLL) return SSM_ERR_SHAPE;
  if (!rows_fit(a->batch, a->channels, a->x_stride) || !rows_fit(a->batch, a->channels, a->r_stride) ||
      !rows_fit(a->batch, a->channels, a->i_stride) || !rows_fit(a->batch, a->channels, a->out_stride) ||
      !product_fits(a->state_slots, a->channels, 1))
    return SSM_ERR_SHAPE;
  if (!io_ok(a->io_dtype)) return SSM_ERR_UNSUPPORTED;
  if (!a->x || !a->r || !a->i || !a->A || !a->state || !a->out) return SSM_ERR_NULL;
  return SSM_OK;
}

namespace {

int norm_common(int64_t rows, int64_t cols, int64_t group, int32_t io, int32_t wide, float eps) {
  if (!positive(rows) || !positive(cols) || !positive(group) || cols % group != 0) return SSM_ERR_SHAPE;
  if (rows > 0x7fffffffLL || cols > 0x7fffffffLL) return SSM_ERR_SHAPE;
  if (!io_ok(io) || (wide != io && wide != SSM_F32) || group > RMS_MAX_GROUP) return SSM_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f)) return SSM_ERR_SHAPE;
  return SSM_OK;
}

}  // namespace

extern "C" int rms_norm_fwd_validate(const rms_norm_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  const int st = norm_common(a->rows, a->cols, a->group_size, a->io_dtype, a->residual_dtype, a->eps);
  if (st != SSM_OK) return st;
  if (!a->x || !a->weight || (!a->residual) != (!a->residual_out)) return SSM_ERR_NULL;
  if ((!a->out && !a->codes) || (!a->codes) != (!a->scales)) return SSM_ERR_NULL;
  if ((a->z && a->residual) || (a->out && a->codes)) return SSM_ERR_UNSUPPORTED;
  if (!rows_fit(a->rows, a->cols, a->x_stride) || (a->z && !rows_fit(a->rows, a->cols, a->z_stride)) ||
      (a->residual && (!rows_fit(a->rows, a->cols, a->residual_stride) || !rows_fit(a->rows, a->cols, a->residual_out_stride))) ||
      (a->out && !rows_fit(a->rows, a->cols, a->out_stride)) || (a->codes && !rows_fit(a->rows, a->cols, a->codes_stride)))
    return SSM_ERR_SHAPE;
  if (a->codes && a->group_size != a->cols && a->group_size % RMS_SCALE_BLOCK != 0) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

extern "C" int rms_norm_bwd_validate(const rms_norm_bwd_args_t *a) {
  if (!a) return SSM_ERR_NULL;
  const int st = norm_common(a->rows, a->cols, a->group_size, a->io_dtype, a->x_dtype, a->eps);
  if (st != SSM_OK) return st;
  if (a->cols / a->group_size > 65535) return SSM_ERR_SHAPE;   // a launch's second dimension
  if (!a->x || !a->weight || !a->dy || !a->dx || !a->dweight || (!a->z) != (!a->dz)) return SSM_ERR_NULL;
  if (a->z && (a->ds || a->dresidual || a->x_dtype != a->io_dtype)) return SSM_ERR_UNSUPPORTED;
  if (!rows_fit(a->rows, a->cols, a->x_stride) || !rows_fit(a->rows, a->cols, a->dy_stride) ||
      !rows_fit(a->rows, a->cols, a->dx_stride) || (a->ds && !rows_fit(a->rows, a->cols, a->ds_stride)) ||
      (a->dresidual && !rows_fit(a->rows, a->cols, a->dresidual_stride)) ||
      (a->z && (!rows_fit(a->rows, a->cols, a->z_stride) || !rows_fit(a->rows, a->cols, a->dz_stride))))
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

extern "C" const char *ssm_status_str(int status) {
  switch (status) {
    case SSM_OK: return "ok";
    case SSM_ERR_NULL: return "a required pointer is NULL";
    case SSM_ERR_SHAPE: return "bad shape (size <= 0, dim not divisible by ngroups, or too large)";
    case SSM_ERR_UNSUPPORTED: return "unsupported argument (dtype, dstate > 16, conv width or cache length out of range, or enum value)";
    case SSM_ERR_HIP: return "HIP runtime error";
    case SSM_ERR_WORKSPACE: return "workspace smaller than required";
    case SSM_ERR_SCRATCH: return "plan needs more scratch than the built-in no-allocation buffer holds";
    default: return "unknown status";
  }
}

extern "C" int ssm_abi_version(void) { return SSM_ABI_VERSION; }
