"""The gated block's operators where they can go wrong.  References and bounds:
gated_ref.py."""
import pytest
import torch

from state_space_model_scan_amd import binding
from tests import gated_ref as R
from tests.harness import log

pytestmark = pytest.mark.gpu
bf, f16, f32, i32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def _randn(g, *shape, dtype=f32, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=i32, device="cuda")


def _cuda(v):
    return None if v is None else v.cuda()


# ---- the norm's eps ---------------------------------------------------------

@pytest.mark.parametrize("io", [f32, bf])
@pytest.mark.parametrize("kind", ["plain", "wide", "gate"])
@pytest.mark.parametrize("eps", [0.0, 1e-12, 0.25])
@pytest.mark.parametrize("T,C,n", [(1, 256, 256), (3, 520, 104), (70, 129, 43), (5, 2560, 2560), (2100, 80, 8), (2, 9001, 9001)])
def test_norm_eps(io, kind, eps, T, C, n):
    """Rows that do not fill a workgroup's units, and eps down to 0."""
    log(f"[norm eps] {io} {kind} {T}x{C} groups of {n} eps {eps}")
    g = torch.Generator().manual_seed(T + C)
    x, w, dy = _randn(g, T, C, dtype=io), 1 + 0.3 * _randn(g, C), _randn(g, T, C, dtype=io)
    z = _randn(g, T, C, dtype=io) if kind == "gate" else None
    res = _randn(g, T, C) if kind == "wide" else None
    ref, err, held = R.norm(x, w, res, z, n, eps)
    got = binding.rms_norm_fwd(x.cuda(), w.cuda(), residual=_cuda(res), z=_cuda(z), group_size=n, eps=eps)
    R.close(got if res is None else got[0], ref, err, io, "out")
    s = x if res is None else held
    want = R.norm_bwd(s, w, dy, z, res, n, eps)
    grads = binding.rms_norm_bwd(s.cuda(), w.cuda(), dy.cuda(), z=_cuda(z), ds=_cuda(res), group_size=n, eps=eps)
    for k, v in grads.items():
        R.close(v, *want[k], {"dweight": f32, "dresidual": f32}.get(k, io), k)


# ---- the weight's gradient of many rows -------------------------------------

@pytest.mark.parametrize("T,C,n,gate", [(200001, 512, 1, False), (100003, 1024, 4, True), (70001, 2048, 64, False)])
def test_norm_weight_gradient_of_many_rows(T, C, n, gate):
    """Terms of one sign whose fp32 sum, one after another, rounds the same way
    each time: 1 + 0.45 2^-11 loses its fraction as long as the sum is between
    2^12 and 2^13."""
    log(f"[norm rows] {T}x{C} groups of {n} gate {gate}")
    g = torch.Generator().manual_seed(C)
    cols = sorted(set(range(2 * n)) | set(range(C - n, C)))
    x = 1 + torch.rand(T, n, generator=g).repeat(1, C // n)
    w, dy = 1 + 0.3 * _randn(g, C), torch.full((T, C), 1 + 0.45 * 2.0 ** -11)
    z = 1 + torch.rand(T, 1, generator=g).expand(T, C) if gate else None
    want = R.norm_bwd(x[:, cols], w[cols], dy[:, cols], None if z is None else z[:, cols], None, n)["dweight"]
    got = binding.rms_norm_bwd(x.cuda(), w.cuda(), dy.cuda(), z=_cuda(z), group_size=n)["dweight"]
    R.close(got[cols], *want, f32, "dweight")
    again = binding.rms_norm_bwd(x.cuda(), w.cuda(), dy.cuda(), z=_cuda(z), group_size=n)["dweight"]
    assert torch.equal(got, again)
