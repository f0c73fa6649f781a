"""Refusals of the packed-token operators: the host checks of the C entry
points and of the Python wrappers, before anything reaches a GPU."""
import ctypes

import pytest
import torch

from state_space_model_scan_amd import _lib, binding

FAKE = 0x1000
bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32


def _conv(**kw):
    a = _lib.ConvVarlenArgs()
    a.total, a.nseq, a.channels, a.width, a.io_dtype, a.act = 10, 2, 24, 4, _lib.SSM_BF16, _lib.SSM_ACT_SILU
    a.x = a.weight = a.cu_seqlens = a.out = a.dout = a.dx = a.dweight = FAKE
    a.x_stride = a.out_stride = a.dout_stride = a.dx_stride = 24
    a.state_slots, a.state_len = 2, 4
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _scan(**kw):
    a = _lib.SsdVarlenArgs()
    a.total, a.nseq, a.max_seqlen, a.nheads, a.headdim, a.dstate, a.ngroups = 100, 2, 60, 4, 64, 128, 2
    a.io_dtype = _lib.SSM_BF16
    a.x = a.dt = a.A = a.B = a.C = a.cu_seqlens = a.out = FAKE
    a.x_stride = a.out_stride = a.z_stride = 256
    a.dt_stride, a.B_stride, a.C_stride, a.state_slots = 4, 256, 256, 2
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _scan_bwd(fwd=None, **kw):
    a = _lib.SsdVarlenBwdArgs()
    a.fwd = _scan(checkpoints=FAKE, checkpoint_scales=FAKE, **(fwd or {}))
    a.dout = a.dx = a.ddt = a.dB = a.dC = a.dA = FAKE
    a.dout_stride = a.dx_stride = a.dB_stride = a.dC_stride = 256
    a.ddt_stride = 4
    a.code_entry_stride, a.code_head_stride, a.scale_entry_stride, a.scale_head_stride = 4 * 64 * 128, 64 * 128, 256, 64
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _step(**kw):
    a = _lib.ConvSsdUpdateArgs()
    a.batch, a.nheads, a.headdim, a.dstate, a.ngroups = 3, 4, 64, 64, 2
    a.io_dtype, a.act, a.width = _lib.SSM_F16, _lib.SSM_ACT_SILU, 4
    a.xBC = a.dt = a.A = a.conv_weight = a.conv_state = a.ssm_state = a.out = FAKE
    a.xBC_stride, a.dt_stride, a.out_stride, a.z_stride, a.state_len, a.state_slots = 512, 4, 256, 256, 4, 3
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _st(name, a):
    return getattr(_lib.lib(), name + "_validate")(ctypes.byref(a))


def test_good_arguments_pass():
    assert _st("causal_conv1d_varlen_fwd", _conv()) == _lib.SSM_OK
    assert _st("causal_conv1d_varlen_fwd", _conv(conv_state=FAKE, state_len=256)) == _lib.SSM_OK
    assert _st("causal_conv1d_varlen_bwd", _conv()) == _lib.SSM_OK
    for n in (32, 64, 128):
        assert _st("ssd_varlen_fwd", _scan(dstate=n)) == _lib.SSM_OK
        assert _st("ssd_varlen_bwd", _scan_bwd(dict(dstate=n))) == _lib.SSM_OK
        assert _st("conv1d_ssd_update", _step(dstate=n, xBC_stride=256 + 4 * n)) == _lib.SSM_OK
    assert _st("ssd_varlen_fwd", _scan(max_seqlen=0, ssm_state=FAKE, z=FAKE)) == _lib.SSM_OK
    assert _lib.lib().ssd_checkpoint_slots(129, 3) == 5 == binding.ssd_checkpoint_slots(129, 3)


N, S, U = _lib.SSM_ERR_NULL, _lib.SSM_ERR_SHAPE, _lib.SSM_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), N), (dict(weight=None), N), (dict(cu_seqlens=None), N), (dict(out=None), N), (dict(total=0), S),
    (dict(nseq=0), S), (dict(channels=0), S), (dict(total=1 << 31), S), (dict(x_stride=23), S), (dict(out_stride=23), S),
    (dict(width=3), U), (dict(io_dtype=7), U), (dict(act=2), U), (dict(conv_state=FAKE, state_len=3), S),
    (dict(conv_state=FAKE, state_len=257), U), (dict(conv_state=FAKE, state_slots=0), S)])
def test_conv_refusals(kw, want):
    assert _st("causal_conv1d_varlen_fwd", _conv(**kw)) == want


@pytest.mark.parametrize("kw,want", [(dict(dout=None), N), (dict(dx=None), N), (dict(dweight=None), N),
                                     (dict(bias=FAKE), N), (dict(dx_stride=1), S), (dict(dout_stride=1), S)])
def test_conv_bwd_refusals(kw, want):
    assert _st("causal_conv1d_varlen_bwd", _conv(**kw)) == want


SCAN_BAD = [(dict(x=None), N), (dict(dt=None), N), (dict(A=None), N), (dict(B=None), N), (dict(C=None), N),
            (dict(cu_seqlens=None), N), (dict(total=0), S), (dict(nseq=0), S), (dict(max_seqlen=101), S),
            (dict(max_seqlen=-1), S), (dict(ngroups=3), S), (dict(headdim=32), U), (dict(dstate=16), U),
            (dict(io_dtype=_lib.SSM_F16), U), (dict(x_stride=255), S), (dict(x_stride=260), U), (dict(B_stride=128), S),
            (dict(x=FAKE + 2), U), (dict(dt_stride=3), S), (dict(dt_limit=1, dt_min=2.0, dt_max=1.0), S),
            (dict(dt_softplus=2), U), (dict(seq_segments=-1), S)]


@pytest.mark.parametrize("kw,want", SCAN_BAD + [
    (dict(out=None), N), (dict(out_stride=255), S), (dict(out=FAKE + 8), U), (dict(z=FAKE, z_stride=0), S),
    (dict(checkpoints=FAKE), N), (dict(checkpoint_scales=FAKE), N), (dict(ssm_state=FAKE, state_slots=0), S),
    (dict(ssm_state=FAKE + 4), U)])
def test_scan_refusals(kw, want):
    assert _st("ssd_varlen_fwd", _scan(**kw)) == want
    size = ctypes.c_size_t()
    assert _lib.lib().ssd_varlen_fwd_workspace_size(ctypes.byref(_scan(**kw)), ctypes.byref(size)) == want


@pytest.mark.parametrize("kw,want", SCAN_BAD + [(dict(z=FAKE), U), (dict(checkpoints=None), N)])
def test_scan_bwd_refuses_the_forwards_arguments(kw, want):
    a = _scan_bwd()
    for k, v in kw.items():
        setattr(a.fwd, k, v)
    assert _st("ssd_varlen_bwd", a) == want


@pytest.mark.parametrize("kw,want", [(dict(dout=None), N), (dict(dx=None), N), (dict(ddt=None), N), (dict(dA=None), N),
                                     (dict(dB=None), N), (dict(dC=None), N), (dict(dx_stride=8), S),
                                     (dict(dx=FAKE + 2), U), (dict(dC_stride=260), U), (dict(ddt_stride=1), S),
                                     (dict(code_entry_stride=64), S), (dict(code_head_stride=64 * 128 + 8), U),
                                     (dict(scale_head_stride=32), S)])
def test_scan_bwd_refusals(kw, want):
    assert _st("ssd_varlen_bwd", _scan_bwd(**kw)) == want


def test_rows_too_far_apart_for_32_bit_offsets_are_refused():
    for key in ("x_stride", "B_stride", "C_stride"):
        for make, name in ((_scan, "ssd_varlen_fwd"), (_scan_bwd, "ssd_varlen_bwd")):
            for stride, want in ((1 << 24, _lib.SSM_OK), ((1 << 24) + 8, S)):
                a = make()
                setattr(a if name == "ssd_varlen_fwd" else a.fwd, key, stride)
                assert _st(name, a) == want
    assert _st("ssd_varlen_bwd", _scan_bwd(dout_stride=1 << 24)) == _lib.SSM_OK
    assert _st("ssd_varlen_bwd", _scan_bwd(dout_stride=(1 << 24) + 8)) == S


def test_scan_bwd_needs_gradients_of_what_is_given():
    for key, grad in (("D", "dD"), ("dt_bias", "ddt_bias")):
        a = _scan_bwd({key: FAKE})
        assert _st("ssd_varlen_bwd", a) == N
        setattr(a, grad, FAKE)
        assert _st("ssd_varlen_bwd", a) == _lib.SSM_OK


@pytest.mark.parametrize("kw,want", [
    (dict(xBC=None), N), (dict(dt=None), N), (dict(conv_state=None), N), (dict(ssm_state=None), N), (dict(out=None), N),
    (dict(batch=0), S), (dict(batch=70000), S), (dict(ngroups=3), S), (dict(headdim=128), U), (dict(dstate=16), U),
    (dict(width=3), U), (dict(io_dtype=9), U), (dict(state_len=3), S), (dict(state_len=300), U), (dict(xBC_stride=511), S),
    (dict(out_stride=1), S), (dict(z=FAKE, z_stride=1), S), (dict(state_slots=0), S), (dict(ssm_state=FAKE + 4), U),
    (dict(dt_limit=1, dt_min=1.0, dt_max=0.0), S)])
def test_step_refusals(kw, want):
    assert _st("conv1d_ssd_update", _step(**kw)) == want


@pytest.mark.parametrize("name,args", [("causal_conv1d_varlen_bwd", _conv), ("ssd_varlen_bwd", _scan_bwd)])
def test_no_workspace(name, args):
    assert getattr(_lib.lib(), name)(ctypes.byref(args()), None) == _lib.SSM_ERR_WORKSPACE


def test_null_arguments():
    L = _lib.lib()
    for name in ("causal_conv1d_varlen_fwd", "causal_conv1d_varlen_bwd", "ssd_varlen_fwd", "ssd_varlen_bwd", "conv1d_ssd_update"):
        assert getattr(L, name)(None, None) == N


# ---- the wrappers ---------------------------------------------------------

T, h, G, n, C = 9, 4, 2, 32, 256 + 128


def _py_conv(**kw):
    t = dict(x=torch.zeros(T, 24, dtype=bf), weight=torch.zeros(24, 4), cu_seqlens=torch.tensor([0, 4, 9], dtype=i32),
             bias=torch.zeros(24), activation="silu")
    t.update(kw)
    return t


def _py_scan(**kw):
    t = dict(x=torch.zeros(T, h, 64, dtype=bf), dt=torch.zeros(T, h, dtype=bf), A=torch.zeros(h),
             B=torch.zeros(T, G, n, dtype=bf), C=torch.zeros(T, G, n, dtype=bf),
             cu_seqlens=torch.tensor([0, 4, 9], dtype=i32), max_seqlen=5)
    t.update(kw)
    return t


def _py_step(**kw):
    t = dict(xBC=torch.zeros(3, C, dtype=bf), dt=torch.zeros(3, h, dtype=bf), A=torch.zeros(h),
             conv_weight=torch.zeros(C, 4), conv_state=torch.zeros(5, C, 4, dtype=bf), ssm_state=torch.zeros(5, h, 64, n),
             cache_seqlens=torch.zeros(3, dtype=i32))
    t.update(kw)
    return t


def test_well_formed_calls_stop_at_the_device_check():
    codes = (torch.zeros(2, h, 64, n, dtype=torch.int8), torch.zeros(2, h, 64))
    for fn, kw in ((binding.causal_conv1d_varlen_fwd, _py_conv()),
                   (binding.causal_conv1d_varlen_bwd, _py_conv(dout=torch.zeros(T, 24, dtype=bf))),
                   (binding.ssd_varlen_fwd, _py_scan(checkpoints=codes)),
                   (binding.ssd_varlen_bwd, _py_scan(checkpoints=codes, dout=torch.zeros(T, h, 64, dtype=bf))),
                   (binding.conv1d_ssd_update, _py_step())):
        with pytest.raises(ValueError, match="cuda device"):
            fn(**kw)


@pytest.mark.parametrize("fn,kw,msg", [
    ("causal_conv1d_varlen_fwd", _py_conv(cu_seqlens=torch.tensor([0, 9])), "cu_seqlens must be torch.int32"),
    ("causal_conv1d_varlen_fwd", _py_conv(cu_seqlens=torch.tensor([0], dtype=i32)), "cu_seqlens must have shape"),
    ("causal_conv1d_varlen_fwd", _py_conv(x=torch.zeros(2, T, 24, dtype=bf)), "x must have 2 dimensions"),
    ("causal_conv1d_varlen_fwd", _py_conv(weight=torch.zeros(23, 4)), "weight must have shape"),
    ("causal_conv1d_varlen_fwd", _py_conv(conv_state=torch.zeros(2, 24, 4)), "conv_state must be torch.bfloat16"),
    ("causal_conv1d_varlen_fwd", _py_conv(slots=torch.zeros(3, dtype=i32)), "slots must have shape"),
    ("causal_conv1d_varlen_bwd", _py_conv(dout=torch.zeros(T, 23, dtype=bf)), "dout must have shape"),
    ("ssd_varlen_fwd", _py_scan(x=torch.zeros(T, h, 64)), "bfloat16"),
    ("ssd_varlen_fwd", _py_scan(max_seqlen=10), "max_seqlen"),
    ("ssd_varlen_fwd", _py_scan(C=torch.zeros(T, G, 64, dtype=bf)), "C must have shape"),
    ("ssd_varlen_fwd", _py_scan(ssm_state=torch.zeros(2, h, n, 64)), "ssm_state must have shape"),
    ("ssd_varlen_fwd", _py_scan(ssm_state=torch.zeros(2, h, n, 64).transpose(2, 3)), "written in place"),
    ("ssd_varlen_fwd", _py_scan(checkpoints=(torch.zeros(1, h, 64, n, dtype=torch.int8), torch.zeros(2, h, 64))),
     "checkpoints"),
    ("ssd_varlen_bwd", _py_scan(dout=torch.zeros(T, h, 64, dtype=bf), checkpoints=None), "needs the checkpoints"),
    ("conv1d_ssd_update", _py_step(xBC=torch.zeros(3, C + 8, dtype=bf)), "xBC must have"),
    ("conv1d_ssd_update", _py_step(conv_state=torch.zeros(4, C, 4, dtype=bf)), "conv_state must have shape"),
    ("conv1d_ssd_update", _py_step(cache_seqlens=torch.zeros(4, dtype=i32)), "cache_seqlens must have shape"),
    ("conv1d_ssd_update", _py_step(z=torch.zeros(3, h, 64, dtype=bf)), "z must have shape")])
def test_wrapper_refusals(fn, kw, msg):
    with pytest.raises(ValueError, match=msg):
        getattr(binding, fn)(**kw)


def test_activation_refusal():
    with pytest.raises(NotImplementedError):
        binding.causal_conv1d_varlen_fwd(**_py_conv(activation="relu"))
