"""Refusals of the gated block's operators: the host checks of the C entry
points and of the Python wrappers, before anything reaches a GPU."""
import ctypes

import pytest
import torch

from state_space_model_scan_amd import _lib, binding

FAKE = 0x1000
bf, f16, f32, i32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
N, S, U = _lib.SSM_ERR_NULL, _lib.SSM_ERR_SHAPE, _lib.SSM_ERR_UNSUPPORTED


def _set(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _scan(**kw):
    a = _lib.GatedScanArgs()
    a.total, a.nseq, a.channels, a.io_dtype = 100, 2, 24, _lib.SSM_BF16
    a.x = a.r = a.i = a.A = a.cu_seqlens = a.out = FAKE
    a.x_stride = a.r_stride = a.i_stride = a.out_stride = 24
    a.state_slots = 3
    return _set(a, kw)


def _scan_bwd(fwd=None, **kw):
    a = _lib.GatedScanBwdArgs()
    a.fwd = _scan(**{**dict(checkpoints=FAKE, out=None), **(fwd or {})})
    a.dout = a.dx = a.dr = a.di = a.dA = FAKE
    a.dout_stride = a.dx_stride = a.dr_stride = a.di_stride = 24
    return _set(a, kw)


def _update(**kw):
    a = _lib.GatedUpdateArgs()
    a.batch, a.channels, a.io_dtype, a.state_slots = 3, 24, _lib.SSM_F16, 4
    a.x = a.r = a.i = a.A = a.state = a.out = FAKE
    a.x_stride = a.r_stride = a.i_stride = a.out_stride = 24
    return _set(a, kw)


def _norm(**kw):
    a = _lib.RmsNormArgs()
    a.rows, a.cols, a.group_size, a.io_dtype, a.residual_dtype, a.eps = 4, 256, 128, _lib.SSM_BF16, _lib.SSM_F32, 1e-5
    a.x = a.weight = a.out = FAKE
    a.x_stride = a.z_stride = a.residual_stride = a.residual_out_stride = a.out_stride = a.codes_stride = 256
    return _set(a, kw)


def _norm_bwd(**kw):
    a = _lib.RmsNormBwdArgs()
    a.rows, a.cols, a.group_size, a.io_dtype, a.x_dtype, a.eps = 4, 256, 128, _lib.SSM_BF16, _lib.SSM_BF16, 1e-5
    a.x = a.weight = a.dy = a.dx = a.dweight = FAKE
    a.x_stride = a.z_stride = a.dy_stride = a.ds_stride = a.dx_stride = a.dresidual_stride = a.dz_stride = 256
    return _set(a, kw)


def _st(name, a):
    return getattr(_lib.lib(), name + "_validate")(ctypes.byref(a))


def test_good_arguments_pass():
    ok = _lib.SSM_OK
    assert _st("gated_scan_varlen_fwd", _scan()) == ok
    assert _st("gated_scan_varlen_fwd", _scan(state=FAKE, checkpoints=FAKE, r_bias=FAKE)) == ok
    assert _st("gated_scan_varlen_bwd", _scan_bwd()) == ok
    assert _st("gated_scan_varlen_bwd", _scan_bwd(dict(r_bias=FAKE, i_bias=FAKE), dr_bias=FAKE, di_bias=FAKE)) == ok
    assert _st("gated_scan_update", _update()) == ok
    assert _st("rms_norm_fwd", _norm()) == ok
    assert _st("rms_norm_fwd", _norm(out=None, codes=FAKE, scales=FAKE, residual=FAKE, residual_out=FAKE)) == ok
    assert _st("rms_norm_fwd", _norm(z=FAKE, eps=0.0)) == ok
    assert _st("rms_norm_bwd", _norm_bwd(z=FAKE, dz=FAKE)) == ok
    assert _st("rms_norm_bwd", _norm_bwd(x_dtype=_lib.SSM_F32, ds=FAKE, dresidual=FAKE)) == ok
    for total in (1, 63, 64, 65, 128, 2 ** 31 - 1):
        assert _lib.lib().gated_checkpoint_slots(total) == binding.gated_checkpoint_slots(total) == (total + 63) // 64


SCAN_BAD = [(dict(x=None), N), (dict(r=None), N), (dict(i=None), N), (dict(A=None), N), (dict(cu_seqlens=None), N),
            (dict(total=0), S), (dict(total=1 << 31), S), (dict(nseq=0), S), (dict(channels=0), S), (dict(channels=1 << 31), S),
            (dict(x_stride=23), S), (dict(r_stride=0), S), (dict(i_stride=-24), S), (dict(x_stride=1 << 60), S),
            (dict(io_dtype=3), U)]


@pytest.mark.parametrize("kw,want", SCAN_BAD + [(dict(out=None), N), (dict(out_stride=23), S),
                                                (dict(state=FAKE, state_slots=0), S),
                                                (dict(state=FAKE, state_slots=1 << 61), S)])
def test_scan_refusals(kw, want):
    assert _st("gated_scan_varlen_fwd", _scan(**kw)) == want
    size = ctypes.c_size_t()
    assert _lib.lib().gated_scan_varlen_fwd_workspace_size(ctypes.byref(_scan(**kw)), ctypes.byref(size)) == want


@pytest.mark.parametrize("kw,want", SCAN_BAD + [(dict(checkpoints=None), N), (dict(r_bias=FAKE), N), (dict(i_bias=FAKE), N)])
def test_scan_bwd_refuses_the_forwards_arguments(kw, want):
    assert _st("gated_scan_varlen_bwd", _scan_bwd(kw)) == want


@pytest.mark.parametrize("kw,want", [(dict(dout=None), N), (dict(dx=None), N), (dict(dr=None), N), (dict(di=None), N),
                                     (dict(dA=None), N), (dict(dout_stride=1), S), (dict(dx_stride=1), S),
                                     (dict(dr_stride=23), S), (dict(di_stride=0), S)])
def test_scan_bwd_refusals(kw, want):
    assert _st("gated_scan_varlen_bwd", _scan_bwd(**kw)) == want
    size = ctypes.c_size_t()
    assert _lib.lib().gated_scan_varlen_bwd_workspace_size(ctypes.byref(_scan_bwd(**kw)), ctypes.byref(size)) == want


@pytest.mark.parametrize("kw,want", [(dict(x=None), N), (dict(r=None), N), (dict(i=None), N), (dict(A=None), N),
                                     (dict(state=None), N), (dict(out=None), N), (dict(batch=0), S), (dict(channels=0), S),
                                     (dict(state_slots=0), S), (dict(x_stride=23), S), (dict(out_stride=1), S),
                                     (dict(io_dtype=9), U), (dict(batch=1 << 31), S)])
def test_update_refusals(kw, want):
    assert _st("gated_scan_update", _update(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), N), (dict(weight=None), N), (dict(out=None), N), (dict(out=None, codes=FAKE), N), (dict(scales=FAKE), N),
    (dict(residual=FAKE), N), (dict(residual_out=FAKE), N), (dict(rows=0), S), (dict(cols=0), S), (dict(group_size=0), S),
    (dict(group_size=100), S), (dict(x_stride=255), S), (dict(z=FAKE, z_stride=1), S), (dict(out_stride=255), S),
    (dict(eps=-1.0), S), (dict(eps=float("nan")), S), (dict(io_dtype=3), U), (dict(residual_dtype=_lib.SSM_F16), U),
    (dict(residual=FAKE, residual_out=FAKE, residual_stride=8), S), (dict(residual=FAKE, residual_out=FAKE, z=FAKE), U),
    (dict(codes=FAKE, scales=FAKE), U), (dict(out=None, codes=FAKE, scales=FAKE, group_size=64), U),
    (dict(out=None, codes=FAKE, scales=FAKE, codes_stride=8), S),
    (dict(cols=32768, group_size=32768, x_stride=32768, out_stride=32768), U)])
def test_norm_refusals(kw, want):
    assert _st("rms_norm_fwd", _norm(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), N), (dict(weight=None), N), (dict(dy=None), N), (dict(dx=None), N), (dict(dweight=None), N),
    (dict(z=FAKE), N), (dict(dz=FAKE), N), (dict(rows=0), S), (dict(group_size=3), S), (dict(dy_stride=2), S),
    (dict(dx_stride=2), S), (dict(ds=FAKE, ds_stride=2), S), (dict(z=FAKE, dz=FAKE, ds=FAKE), U),
    (dict(z=FAKE, dz=FAKE, x_dtype=_lib.SSM_F32), U), (dict(x_dtype=_lib.SSM_F16), U), (dict(z=FAKE, dz=FAKE, dz_stride=2), S)])
def test_norm_bwd_refusals(kw, want):
    assert _st("rms_norm_bwd", _norm_bwd(**kw)) == want
    size = ctypes.c_size_t()
    assert _lib.lib().rms_norm_bwd_workspace_size(ctypes.byref(_norm_bwd(**kw)), ctypes.byref(size)) == want


# ---- the wrappers -----------------------------------------------------------

def _scan_tensors(T=70, C=24, io=bf, s=2):
    return dict(x=torch.zeros(T, C, dtype=io), r=torch.zeros(T, C, dtype=io), i=torch.zeros(T, C, dtype=io), A=torch.zeros(C),
                cu_seqlens=torch.zeros(s + 1, dtype=i32))


WRONG = [("x", torch.zeros(70, 24, dtype=torch.float64), "io dtype"), ("x", torch.zeros(70, dtype=bf), "2 dimensions"),
         ("r", torch.zeros(70, 23, dtype=bf), "r must have shape"), ("r", torch.zeros(70, 24), "r must be"),
         ("i", torch.zeros(69, 24, dtype=bf), "i must have shape"), ("i", torch.zeros(70, 24, dtype=f16), "i must be"),
         ("A", torch.zeros(25), "A must have shape"), ("A", torch.zeros(24, dtype=bf), "A must be"),
         ("r_bias", torch.zeros(23), "r_bias"), ("i_bias", torch.zeros(24, dtype=bf), "i_bias"),
         ("x", torch.zeros(70, 24, dtype=bf, device="meta"), "must be on meta")]
CU = [("cu_seqlens", torch.zeros(1, dtype=i32), "cu_seqlens"), ("cu_seqlens", torch.zeros(3, dtype=torch.int64), "cu_seqlens")]


@pytest.mark.parametrize("name,value,text", WRONG + CU + [
    ("state", torch.zeros(3, 23), "state"), ("state", torch.zeros(3, 24, 1), "state must have shape"),
    ("state", torch.zeros(24, 3).t(), "contiguous"), ("state", torch.zeros(3, 24, dtype=bf), "state must be"),
    ("cache_seqlens", torch.zeros(3, dtype=i32), "cache_seqlens"), ("slots", torch.zeros(2), "slots"),
    ("checkpoints", torch.zeros(1, 24), "checkpoints"), ("out", torch.zeros(70, 24), "GPU")])
def test_scan_wrapper_refuses(name, value, text):
    with pytest.raises(ValueError, match=text):
        binding.gated_scan_varlen_fwd(**{**_scan_tensors(), name: value})


@pytest.mark.parametrize("name,value,text", WRONG + CU + [
    ("dout", torch.zeros(70, 24), "dout"), ("checkpoints", torch.zeros(2, 23), "checkpoints"), ("checkpoints", None, "checkpoints"),
    ("initial_states", torch.zeros(3, 24), "initial_states"), ("dfinal_states", torch.zeros(2, 24, dtype=bf), "dfinal_states")])
def test_scan_bwd_wrapper_refuses(name, value, text):
    kw = dict(_scan_tensors(), dout=torch.zeros(70, 24, dtype=bf), checkpoints=torch.zeros(2, 24))
    with pytest.raises(ValueError, match=text):
        binding.gated_scan_varlen_bwd(**{**kw, name: value})


@pytest.mark.parametrize("name,value,text", WRONG + [
    ("state", torch.zeros(3, 23), "state"), ("cache_seqlens", torch.zeros(69, dtype=i32), "cache_seqlens"),
    ("slots", torch.zeros(70, dtype=torch.int64), "slots")])
def test_update_wrapper_refuses(name, value, text):
    kw = dict(_scan_tensors(), state=torch.zeros(80, 24), cache_seqlens=torch.zeros(70, dtype=i32))
    del kw["cu_seqlens"]
    with pytest.raises(ValueError, match=text):
        binding.gated_scan_update(**{**kw, name: value})


def _norm_tensors():
    return dict(x=torch.zeros(4, 256, dtype=bf), weight=torch.zeros(256))


@pytest.mark.parametrize("name,value,text", [
    ("x", torch.zeros(4, 256, dtype=torch.int32), "io dtype"), ("weight", torch.zeros(255), "weight"),
    ("weight", torch.zeros(256, dtype=bf), "weight"), ("z", torch.zeros(4, 256), "z must be"),
    ("residual", torch.zeros(4, 256, dtype=f16), "residual must be"), ("residual", torch.zeros(4, 255), "residual must have"),
    ("residual_out", torch.zeros(4, 256), "goes with a residual")])
@pytest.mark.parametrize("fn", ["rms_norm_fwd", "rms_norm_quant_fwd"])
def test_norm_wrapper_refuses(fn, name, value, text):
    with pytest.raises(ValueError, match=text):
        getattr(binding, fn)(**{**_norm_tensors(), name: value})
    with pytest.raises(ValueError, match="not both"):
        getattr(binding, fn)(**_norm_tensors(), residual=torch.zeros(4, 256), z=torch.zeros(4, 256, dtype=bf))
    with pytest.raises(ValueError, match="GPU"):
        getattr(binding, fn)(**_norm_tensors())


def test_norm_quant_wrapper_refuses():
    with pytest.raises(ValueError, match="scales"):
        binding.rms_norm_quant_fwd(**_norm_tensors(), scales=torch.zeros(4, 1))


@pytest.mark.parametrize("name,value,text", [
    ("x", torch.zeros(4, 256, dtype=f16), "x must be"), ("dy", torch.zeros(4, 255, dtype=bf), "x must have"),
    ("weight", torch.zeros(4), "weight"), ("z", torch.zeros(4, 256), "z must be"), ("ds", torch.zeros(4, 256), "ds must be"),
    ("dz", torch.zeros(4, 256, dtype=bf), "dz goes with z"), ("dresidual", torch.zeros(4, 256, dtype=bf), "dresidual goes with")])
def test_norm_bwd_wrapper_refuses(name, value, text):
    kw = dict(_norm_tensors(), dy=torch.zeros(4, 256, dtype=bf))
    with pytest.raises(ValueError, match=text):
        binding.rms_norm_bwd(**{**kw, name: value})
    with pytest.raises(ValueError, match="not both"):
        binding.rms_norm_bwd(**kw, z=kw["x"], ds=kw["x"])
    with pytest.raises(ValueError, match="one dtype"):
        binding.rms_norm_bwd(torch.zeros(4, 256), kw["weight"], kw["dy"], z=kw["x"])


def test_norm_bwd_refuses_more_groups_than_a_launch_takes():
    wide = {k + "_stride": 65536 for k in ("x", "z", "dy", "ds", "dx", "dresidual", "dz")}
    assert _st("rms_norm_bwd", _norm_bwd(cols=65536, group_size=1, **wide)) == S
    assert _st("rms_norm_bwd", _norm_bwd(cols=65535, group_size=1, **wide)) == _lib.SSM_OK


def test_scans_refuse_a_workspace_off_16_bytes():
    """... and one that is too small or missing, before anything is launched."""
    L, size = _lib.lib(), ctypes.c_size_t()
    for make, name in ((lambda **kw: _scan(total=1000, **kw), "gated_scan_varlen_fwd"),
                       (lambda **kw: _scan_bwd(dict(total=1000), **kw), "gated_scan_varlen_bwd")):
        assert getattr(L, name + "_workspace_size")(ctypes.byref(make()), ctypes.byref(size)) == _lib.SSM_OK and size.value > 0
        for kw, want in ((dict(), _lib.SSM_ERR_WORKSPACE), (dict(workspace=FAKE, workspace_bytes=size.value - 1), _lib.SSM_ERR_WORKSPACE),
                         (dict(workspace=FAKE + 8, workspace_bytes=size.value), U)):
            assert getattr(L, name)(ctypes.byref(make(**kw)), None) == want, (name, kw)
