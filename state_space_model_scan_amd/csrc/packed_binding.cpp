// packed_binding.cpp -- the torch binding of the packed-token operators
// (module _packed).  Argument checks and marshalling only: every step of an
// operator runs in libssmscan's kernels behind the C ABI.
//
// Their smallest calls take the GPU about five microseconds, which is less
// than the same checks take in Python (16 to 48 us a call).  Each function
// returns (status, outputs...); binding.py names the arguments, documents them
// and turns a status into an exception.  A refused tensor raises ValueError
// with the text that the other wrappers use.
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ATen.h>

#include <optional>
#include <sstream>
#include <string>
#include <tuple>

#include "ssmscan.h"

namespace py = pybind11;
using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;
using Opt = std::optional<Tensor>;

namespace {

[[noreturn]] void refuse(const std::string &text) { throw py::value_error(text); }

std::string tuple_text(IntArrayRef v) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < v.size(); ++i) s << (i ? ", " : "") << v[i];
  s << (v.size() == 1 ? ",)" : ")");
  return s.str();
}

std::string dtype_text(ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kChar: return "torch.int8";
    case at::kDouble: return "torch.float64";
    default: return c10::toString(t);
  }
}

void spec(const Tensor &t, const char *name, IntArrayRef shape, ScalarType dtype, at::Device dev) {
  if (t.sizes() == shape && t.scalar_type() == dtype && t.device() == dev) return;
  std::ostringstream s;
  if (t.sizes() != shape) s << name << " must have shape " << tuple_text(shape) << ", got " << tuple_text(t.sizes());
  else if (t.scalar_type() != dtype) s << name << " must be " << dtype_text(dtype) << ", got " << dtype_text(t.scalar_type());
  else s << name << " must be on " << dev << " with the other tensors, got " << t.device();
  refuse(s.str());
}
void spec(const Opt &t, const char *name, IntArrayRef shape, ScalarType dtype, at::Device dev) {
  if (t) spec(*t, name, shape, dtype, dev);
}
void out_spec(const Opt &t, const char *name, IntArrayRef shape, ScalarType dtype, at::Device dev) {
  spec(t, name, shape, dtype, dev);
  if (t && !t->is_contiguous()) refuse(std::string(name) + " is written in place and must be contiguous");
}
void on_gpu(at::Device dev) {
  if (!dev.is_cuda()) refuse("the operator runs on the GPU: tensors must be on a cuda device, got " + dev.str());
}
int io_of(const Tensor &t, const char *name, int64_t ndim) {
  const int io = t.scalar_type() == at::kFloat ? SSM_F32 : t.scalar_type() == at::kBFloat16 ? SSM_BF16
                 : t.scalar_type() == at::kHalf ? SSM_F16 : -1;
  if (io < 0) refuse("io dtype must be float32, bfloat16 or float16, got " + dtype_text(t.scalar_type()));
  if (t.dim() != ndim)
    refuse(std::string(name) + " must have " + std::to_string(ndim) + " dimensions, got shape " + tuple_text(t.sizes()));
  return io;
}

Tensor dense(const Tensor &t) { return t.contiguous(); }
Opt dense(const Opt &t) { return t ? Opt(t->contiguous()) : Opt(); }
// ... and 16-byte aligned
Opt dense16(const Opt &t) {
  if (!t) return {};
  const Tensor d = t->contiguous();
  return reinterpret_cast<uintptr_t>(d.data_ptr()) % 16 == 0 ? d : d.clone();
}

// t as the library takes a packed tensor: whatever a token holds dense, any
// stride from token to token; with vec, the first element 16-byte aligned and
// the stride a multiple of vec elements.
bool fits(const Tensor &t, int64_t vec) {
  int64_t want = 1;
  for (int64_t d = t.dim() - 1; d > 0; --d) {
    if (t.stride(d) != want && t.size(d) != 1) return false;
    want *= t.size(d);
  }
  if (t.size(0) > 1 && (t.stride(0) < want || (vec && t.stride(0) % vec))) return false;
  return !vec || (want % vec == 0 && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0);
}
Tensor tokens(const Tensor &t, int64_t vec = 0) {
  return fits(t, vec) ? t : t.clone(at::MemoryFormat::Contiguous);
}
Opt tokens(const Opt &t, int64_t vec = 0) { return t ? Opt(tokens(*t, vec)) : Opt(); }
int64_t stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.numel(); }

Tensor make(IntArrayRef shape, ScalarType dtype, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}
// an output given by the caller (checked) or a new one
Tensor tokens_out(const Opt &t, const char *name, IntArrayRef shape, ScalarType dtype, at::Device dev, int64_t vec = 0) {
  if (!t) return make(shape, dtype, dev);
  spec(*t, name, shape, dtype, dev);
  if (!fits(*t, vec)) {
    std::string s = std::string(name) + " is written in place: what a token holds must be dense";
    if (vec) s += ", its start 16-byte aligned and its token stride a multiple of " + std::to_string(vec);
    refuse(s);
  }
  return *t;
}

const void *addr(const Tensor &t) { return t.data_ptr(); }
const float *f32(const Tensor &t) { return t.data_ptr<float>(); }
const float *f32(const Opt &t) { return t ? t->data_ptr<float>() : nullptr; }
const int32_t *i32(const Opt &t) { return t ? t->data_ptr<int32_t>() : nullptr; }

int64_t cu_spec(const Tensor &cu, at::Device dev) {
  if (cu.dim() != 1 || cu.size(0) < 2)
    refuse("cu_seqlens must have shape (nseq + 1,) with nseq >= 1, got " + tuple_text(cu.sizes()));
  spec(cu, "cu_seqlens", cu.sizes(), at::kInt, dev);
  return cu.size(0) - 1;
}

void conv_params(const Tensor &w, const Opt &bias, int64_t channels, at::Device dev) {
  if (w.dim() != 2) refuse("conv weight must be (dim, width), got shape " + tuple_text(w.sizes()));
  spec(w, "weight", {channels, w.size(1)}, at::kFloat, dev);
  spec(bias, "bias", {channels}, at::kFloat, dev);
}

// The stream of a call, for as long as the call lasts: one that the caller
// names becomes torch's current one, so that the copies of inputs, the
// workspace and new outputs are made on it, in order with the kernels, and
// memory that the call gives back is not handed out to another stream.
class OnStream {
 public:
  OnStream(at::Device dev, std::optional<int64_t> given) : dev_(dev) {
    if (!given || !dev.is_cuda()) return;
    before_ = c10::hip::getCurrentHIPStream(dev.index());
    c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal(reinterpret_cast<hipStream_t>(*given), dev.index()));
  }
  ~OnStream() {
    if (before_) c10::hip::setCurrentHIPStream(*before_);
  }
  OnStream(const OnStream &) = delete;
  OnStream &operator=(const OnStream &) = delete;
  void *handle() const { return c10::hip::getCurrentHIPStream(dev_.index()).stream(); }

 private:
  at::Device dev_;
  std::optional<c10::hip::HIPStream> before_;
};

// the caller's scratch, or as much as the call needs
template <typename Args>
int workspace(int (*size)(const Args *, size_t *), Args &a, const Opt &given, at::Device dev, Opt &held) {
  held = given;
  if (!given) {
    size_t need = 0;
    if (const int st = size(&a, &need)) return st;
    if (need) held = make({static_cast<int64_t>(need)}, at::kByte, dev);
  } else if (given->device() != dev || !given->is_contiguous()) {
    refuse("workspace must be a contiguous tensor on " + dev.str());
  }
  if (held) {
    a.workspace = held->data_ptr();
    a.workspace_bytes = held->nbytes();
  }
  return SSM_OK;
}

// ---------------------------------------------------------------------------

struct Conv {
  Tensor x, w, cu;
  Opt bias;
  causal_conv1d_varlen_args_t a{};

  Conv(const Tensor &x_, const Tensor &w_, const Tensor &cu_, const Opt &bias_, int act) {
    a.io_dtype = io_of(x_, "x", 2);
    const at::Device dev = x_.device();
    conv_params(w_, bias_, x_.size(1), dev);
    a.nseq = cu_spec(cu_, dev);
    x = tokens(x_);
    w = dense(w_);
    cu = dense(cu_);
    bias = dense(bias_);
    a.total = x.size(0);
    a.channels = x.size(1);
    a.width = static_cast<int32_t>(w.size(1));
    a.act = act;
    a.x = addr(x);
    a.x_stride = stride(x);
    a.weight = f32(w);
    a.bias = f32(bias);
    a.cu_seqlens = cu.data_ptr<int32_t>();
  }
};

std::tuple<int, Tensor> conv_fwd(const Tensor &x, const Tensor &w, const Tensor &cu, const Opt &bias, int act,
                                 const Opt &conv_state, const Opt &seen_, const Opt &slots_, const Opt &out_,
                                 std::optional<int64_t> stream) {
  const at::Device dev = x.device();
  const OnStream on(dev, stream);
  Conv c(x, w, cu, bias, act);
  spec(seen_, "cache_seqlens", {c.a.nseq}, at::kInt, dev);
  spec(slots_, "slots", {c.a.nseq}, at::kInt, dev);
  if (conv_state) {
    if (conv_state->dim() != 3)
      refuse("conv_state must have shape (entries, channels, state_len), got " + tuple_text(conv_state->sizes()));
    out_spec(conv_state, "conv_state", {conv_state->size(0), x.size(1), conv_state->size(2)}, x.scalar_type(), dev);
    c.a.conv_state = conv_state->data_ptr();
    c.a.state_slots = conv_state->size(0);
    c.a.state_len = conv_state->size(2);
  }
  on_gpu(dev);
  const Tensor out = tokens_out(out_, "out", x.sizes(), x.scalar_type(), dev);
  const Opt seen = dense(seen_), slots = dense(slots_);
  c.a.out = out.data_ptr();
  c.a.out_stride = stride(out);
  c.a.cache_seqlens = i32(seen);
  c.a.slots = i32(slots);
  return {causal_conv1d_varlen_fwd(&c.a, on.handle()), out};
}

std::tuple<int, Tensor, Tensor, Opt> conv_bwd(const Tensor &x, const Tensor &w, const Tensor &cu, const Tensor &dout_,
                                              const Opt &bias, int act, const Opt &dx_, const Opt &ws_,
                                              std::optional<int64_t> stream) {
  const at::Device dev = x.device();
  const OnStream on(dev, stream);
  Conv c(x, w, cu, bias, act);
  spec(dout_, "dout", x.sizes(), x.scalar_type(), dev);
  on_gpu(dev);
  const Tensor dout = tokens(dout_), dx = tokens_out(dx_, "dx", x.sizes(), x.scalar_type(), dev);
  const Tensor dw = make(w.sizes(), at::kFloat, dev);
  Opt db;
  if (bias) db = make(bias->sizes(), at::kFloat, dev);
  c.a.dout = addr(dout);
  c.a.dout_stride = stride(dout);
  c.a.dx = dx.data_ptr();
  c.a.dx_stride = stride(dx);
  c.a.dweight = dw.data_ptr<float>();
  c.a.dbias = db ? db->data_ptr<float>() : nullptr;
  Opt ws;
  int st = workspace(causal_conv1d_varlen_bwd_workspace_size, c.a, ws_, dev, ws);
  if (st == SSM_OK) st = causal_conv1d_varlen_bwd(&c.a, on.handle());
  return {st, dx, dw, db};
}

struct Scan {
  Tensor x, dt, A, B, C, cu;
  Opt D, z, dt_bias, codes, scales;
  ssd_varlen_args_t a{};

  Scan(const Tensor &x_, const Tensor &dt_, const Tensor &A_, const Tensor &B_, const Tensor &C_, const Tensor &cu_,
       int64_t max_seqlen, const Opt &D_, const Opt &z_, const Opt &dt_bias_, bool softplus,
       std::optional<std::tuple<double, double>> limit, const Opt &codes_, const Opt &scales_, int64_t segments) {
    const ScalarType io = x_.scalar_type(), f = at::kFloat;
    if (io != at::kBFloat16) refuse("the packed scan takes bfloat16 io, got " + dtype_text(io));
    if (x_.dim() != 3 || B_.dim() != 3) refuse("x must be (total, nheads, headdim) and B (total, ngroups, dstate)");
    const int64_t total = x_.size(0), h = x_.size(1), p = x_.size(2), g = B_.size(1), n = B_.size(2);
    const at::Device dev = x_.device();
    spec(z_, "z", x_.sizes(), io, dev);
    spec(dt_, "dt", {total, h}, io, dev);
    spec(B_, "B", {total, g, n}, io, dev);
    spec(C_, "C", {total, g, n}, io, dev);
    spec(A_, "A", {h}, f, dev);
    spec(dt_bias_, "dt_bias", {h}, f, dev);
    if (D_ && D_->dim() == 1) spec(D_, "D", {h}, f, dev);
    else spec(D_, "D", {h, p}, f, dev);
    a.nseq = cu_spec(cu_, dev);
    if (max_seqlen < 0 || max_seqlen > total)
      refuse("max_seqlen must be the longest sequence's length, at most " + std::to_string(total) + ", got " +
             std::to_string(max_seqlen));
    if (codes_.has_value() != scales_.has_value()) refuse("checkpoints must be the codes and their scales, got one of them");
    if (codes_) {
      const int64_t e = ssd_checkpoint_slots(total, a.nseq);
      spec(codes_, "checkpoints[0]", {e, h, p, n}, at::kChar, dev);
      spec(scales_, "checkpoints[1]", {e, h, p}, f, dev);
    }
    x = tokens(x_, 8); B = tokens(B_, 8); C = tokens(C_, 8); z = tokens(z_, 8); dt = tokens(dt_);
    A = dense(A_); D = dense(D_); dt_bias = dense(dt_bias_); cu = dense(cu_);
    codes = codes_; scales = scales_;
    a.total = total; a.max_seqlen = max_seqlen;
    a.nheads = h; a.headdim = p; a.dstate = n; a.ngroups = g; a.io_dtype = SSM_BF16;
    a.x = addr(x); a.x_stride = stride(x);
    a.dt = addr(dt); a.dt_stride = stride(dt);
    a.A = f32(A);
    a.B = addr(B); a.B_stride = stride(B);
    a.C = addr(C); a.C_stride = stride(C);
    a.D = f32(D); a.D_per_channel = D && D->dim() == 2;
    if (z) { a.z = addr(*z); a.z_stride = stride(*z); }
    a.dt_bias = f32(dt_bias);
    a.dt_softplus = softplus;
    if (limit) { a.dt_limit = 1; a.dt_min = static_cast<float>(std::get<0>(*limit)); a.dt_max = static_cast<float>(std::get<1>(*limit)); }
    a.cu_seqlens = cu.data_ptr<int32_t>();
    a.seq_segments = static_cast<int32_t>(segments);
    if (codes) { a.checkpoints = codes->data_ptr<int8_t>(); a.checkpoint_scales = scales->data_ptr<float>(); }
  }
};

std::tuple<int, Tensor> scan_fwd(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &B, const Tensor &C,
                                 const Tensor &cu, int64_t max_seqlen, const Opt &D, const Opt &z, const Opt &dt_bias,
                                 bool softplus, std::optional<std::tuple<double, double>> limit, const Opt &state,
                                 const Opt &seen_, const Opt &slots_, const Opt &codes, const Opt &scales, const Opt &out_,
                                 const Opt &ws_, int64_t segments, std::optional<int64_t> stream) {
  const at::Device dev = x.device();
  const OnStream on(dev, stream);
  Scan s(x, dt, A, B, C, cu, max_seqlen, D, z, dt_bias, softplus, limit, codes, scales, segments);
  if (state) {
    if (state->dim() != 4)
      refuse("ssm_state must have shape (entries, nheads, headdim, dstate), got " + tuple_text(state->sizes()));
    out_spec(state, "ssm_state", {state->size(0), s.a.nheads, s.a.headdim, s.a.dstate}, at::kFloat, dev);
    s.a.ssm_state = state->data_ptr<float>();
    s.a.state_slots = state->size(0);
  }
  spec(seen_, "cache_seqlens", {s.a.nseq}, at::kInt, dev);
  spec(slots_, "slots", {s.a.nseq}, at::kInt, dev);
  if (codes) {
    out_spec(codes, "checkpoints[0]", codes->sizes(), at::kChar, dev);
    out_spec(scales, "checkpoints[1]", scales->sizes(), at::kFloat, dev);
  }
  on_gpu(dev);
  const Tensor out = tokens_out(out_, "out", x.sizes(), x.scalar_type(), dev, 8);
  const Opt seen = dense(seen_), slots = dense(slots_);
  s.a.out = out.data_ptr();
  s.a.out_stride = stride(out);
  s.a.cache_seqlens = i32(seen);
  s.a.slots = i32(slots);
  Opt ws;
  int st = workspace(ssd_varlen_fwd_workspace_size, s.a, ws_, dev, ws);
  if (st == SSM_OK) st = ssd_varlen_fwd(&s.a, on.handle());
  return {st, out};
}

using BwdOut = std::tuple<int, Tensor, Tensor, Tensor, Tensor, Tensor, Opt, Opt, Opt>;

BwdOut scan_bwd(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &B, const Tensor &C, const Tensor &cu,
                int64_t max_seqlen, const Tensor &dout_, const Tensor &codes_, const Tensor &scales_, const Opt &D,
                const Opt &dt_bias, bool softplus, std::optional<std::tuple<double, double>> limit, const Opt &dfin_,
                bool want_init, const Opt &dx_, const Opt &dB_, const Opt &dC_, const Opt &ddt_, const Opt &ws_,
                int64_t segments, std::optional<int64_t> stream) {
  const at::Device dev = x.device();
  const OnStream on(dev, stream);
  ssd_varlen_bwd_args_t a{};
  Scan s(x, dt, A, B, C, cu, max_seqlen, D, {}, dt_bias, softplus, limit, codes_, scales_, segments);
  const ScalarType io = x.scalar_type(), f = at::kFloat;
  const int64_t h = s.a.nheads, p = s.a.headdim, n = s.a.dstate;
  // any strides from entry to entry and head to head; a channel's states dense
  Tensor codes = codes_, scales = scales_;
  if (codes.stride(3) != 1 || codes.stride(2) != n || codes.stride(0) % 16 || codes.stride(1) % 16 ||
      std::min(codes.stride(0), codes.stride(1)) < p * n || reinterpret_cast<uintptr_t>(codes.data_ptr()) % 16)
    codes = codes.clone(at::MemoryFormat::Contiguous);
  if (scales.stride(2) != 1 || std::min(scales.stride(0), scales.stride(1)) < p)
    scales = scales.clone(at::MemoryFormat::Contiguous);
  s.a.checkpoints = codes.data_ptr<int8_t>();
  s.a.checkpoint_scales = scales.data_ptr<float>();
  spec(dout_, "dout", x.sizes(), io, dev);
  spec(dfin_, "dfinal_states", {s.a.nseq, h, p, n}, f, dev);
  const Tensor dout = tokens(dout_, 8);
  const Opt dfin = dense16(dfin_);
  on_gpu(dev);
  const Tensor dx = tokens_out(dx_, "dx", x.sizes(), io, dev, 8), ddt = tokens_out(ddt_, "ddt", dt.sizes(), io, dev);
  const Tensor dB = tokens_out(dB_, "dB", B.sizes(), io, dev, 8), dC = tokens_out(dC_, "dC", C.sizes(), io, dev, 8);
  const Tensor dA = make({h}, f, dev);
  Opt dD, db, dinit;
  if (D) dD = make(D->sizes(), f, dev);
  if (dt_bias) db = make({h}, f, dev);
  if (want_init) dinit = make({s.a.nseq, h, p, n}, f, dev);
  a.fwd = s.a;
  a.code_entry_stride = codes.stride(0); a.code_head_stride = codes.stride(1);
  a.scale_entry_stride = scales.stride(0); a.scale_head_stride = scales.stride(1);
  a.dout = addr(dout); a.dout_stride = stride(dout);
  a.dfinal_states = f32(dfin);
  a.dx = dx.data_ptr(); a.dx_stride = stride(dx);
  a.ddt = ddt.data_ptr(); a.ddt_stride = stride(ddt);
  a.dB = dB.data_ptr(); a.dB_stride = stride(dB);
  a.dC = dC.data_ptr(); a.dC_stride = stride(dC);
  a.dA = dA.data_ptr<float>();
  a.dD = dD ? dD->data_ptr<float>() : nullptr;
  a.ddt_bias = db ? db->data_ptr<float>() : nullptr;
  a.dinitial_states = dinit ? dinit->data_ptr<float>() : nullptr;
  Opt ws;
  int st = workspace(ssd_varlen_bwd_workspace_size, a, ws_, dev, ws);
  if (st == SSM_OK) st = ssd_varlen_bwd(&a, on.handle());
  return {st, dx, ddt, dB, dC, dA, dD, db, dinit};
}

std::tuple<int, Tensor> step(const Tensor &xBC_, const Tensor &dt_, const Tensor &A_, const Tensor &w_, const Tensor &ring,
                             const Tensor &state, const Opt &seen_, const Opt &wb_, const Opt &D_, const Opt &z_,
                             const Opt &dt_bias_, bool softplus, std::optional<std::tuple<double, double>> limit,
                             const Opt &slots_, int act, const Opt &out_, std::optional<int64_t> stream) {
  conv1d_ssd_update_args_t a{};
  a.io_dtype = io_of(xBC_, "xBC", 2);
  const ScalarType io = xBC_.scalar_type(), f = at::kFloat;
  const at::Device dev = xBC_.device();
  const OnStream on(dev, stream);
  if (state.dim() != 4)
    refuse("ssm_state must be (entries, nheads, headdim, dstate), got shape " + tuple_text(state.sizes()));
  const int64_t e = state.size(0), h = state.size(1), p = state.size(2), n = state.size(3), hp = h * p;
  const int64_t batch = xBC_.size(0), channels = xBC_.size(1);
  if (n < 1 || channels <= hp || (channels - hp) % (2 * n) != 0)
    refuse("xBC must have nheads * headdim + 2 * ngroups * dstate columns, got " + std::to_string(channels) + " for " +
           std::to_string(h) + " heads of " + std::to_string(p) + " and dstate " + std::to_string(n));
  out_spec(state, "ssm_state", state.sizes(), f, dev);
  if (ring.dim() != 3) refuse("conv_state must be (entries, channels, state_len), got shape " + tuple_text(ring.sizes()));
  out_spec(ring, "conv_state", {e, channels, ring.size(2)}, io, dev);
  conv_params(w_, wb_, channels, dev);
  spec(dt_, "dt", {batch, h}, io, dev);
  spec(z_, "z", {batch, hp}, io, dev);
  spec(A_, "A", {h}, f, dev);
  spec(dt_bias_, "dt_bias", {h}, f, dev);
  if (D_ && D_->dim() == 1) spec(D_, "D", {h}, f, dev);
  else spec(D_, "D", {h, p}, f, dev);
  spec(seen_, "cache_seqlens", {batch}, at::kInt, dev);
  spec(slots_, "slots", {batch}, at::kInt, dev);
  on_gpu(dev);
  const Tensor out = tokens_out(out_, "out", {batch, hp}, io, dev);
  const Tensor xBC = tokens(xBC_), dt = tokens(dt_), A = dense(A_), w = dense(w_);
  const Opt z = tokens(z_), wb = dense(wb_), D = dense(D_), dt_bias = dense(dt_bias_), seen = dense(seen_), slots = dense(slots_);
  a.batch = batch; a.nheads = h; a.headdim = p; a.dstate = n; a.ngroups = (channels - hp) / (2 * n);
  a.act = act; a.width = static_cast<int32_t>(w.size(1));
  a.xBC = addr(xBC); a.xBC_stride = stride(xBC);
  a.dt = addr(dt); a.dt_stride = stride(dt);
  a.A = f32(A); a.conv_weight = f32(w); a.conv_bias = f32(wb);
  a.D = f32(D); a.D_per_channel = D && D->dim() == 2;
  if (z) { a.z = addr(*z); a.z_stride = stride(*z); }
  a.dt_bias = f32(dt_bias);
  a.dt_softplus = softplus;
  if (limit) { a.dt_limit = 1; a.dt_min = static_cast<float>(std::get<0>(*limit)); a.dt_max = static_cast<float>(std::get<1>(*limit)); }
  a.conv_state = ring.data_ptr(); a.state_len = ring.size(2);
  a.ssm_state = state.data_ptr<float>(); a.state_slots = e;
  a.cache_seqlens = i32(seen); a.slots = i32(slots);
  a.out = out.data_ptr(); a.out_stride = stride(out);
  return {conv1d_ssd_update(&a, on.handle()), out};
}

}  // namespace

PYBIND11_MODULE(_packed, m) {
  m.doc() = "Checks and marshalling of the packed-token operators (see binding.py).";
  m.def("conv_fwd", &conv_fwd);
  m.def("conv_bwd", &conv_bwd);
  m.def("scan_fwd", &scan_fwd);
  m.def("scan_bwd", &scan_bwd);
  m.def("step", &step);
}
