"""The 64-bit references of the gated block's operators against torch's own
differentiation and against differences."""
import torch

from tests import gated_ref as R

f64 = torch.float64


def _case(lens, C, seed=0, first=0, tail=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + first + tail
    rand = lambda *s: torch.randn(s, generator=g, dtype=f64)  # noqa: E731
    t = dict(x=rand(T, C), r=rand(T, C), i=rand(T, C), A=-8 * torch.rand(C, generator=g, dtype=f64) * 0.3, r_bias=rand(C),
             i_bias=rand(C))
    return t, R.sequences(lens, first), rand


def _loss(t, cu, h0, dout, dfin):
    total = 0.0
    for s in range(len(cu) - 1):
        h = h0[s]
        for k in range(cu[s], cu[s + 1]):
            a = torch.exp(t["A"] * torch.sigmoid(t["r"][k] + t["r_bias"]))
            h = a * h + torch.sqrt(1 - a * a) * torch.sigmoid(t["i"][k] + t["i_bias"]) * t["x"][k]
            total = total + (h * dout[k]).sum()
        total = total + (h * dfin[s]).sum()
    return total


def test_scan_gradients_are_the_formulas():
    t, cu, rand = _case((5, 0, 1, 9), 3, first=2, tail=1)
    h0, dfin, dout = rand(4, 3), rand(4, 3), rand(18, 3)
    leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
    start = h0.clone().requires_grad_()
    _loss(leaves, cu, start, dout, dfin).backward()
    got = R.scan_bwd(t, cu, dout, h0, dfin)
    for name, leaf in (("dx", "x"), ("dr", "r"), ("di", "i"), ("dA", "A"), ("dr_bias", "r_bias"), ("di_bias", "i_bias")):
        assert torch.allclose(got[name][0], leaves[leaf].grad, rtol=1e-10, atol=1e-12), name
    assert torch.allclose(got["dinitial_states"][0], start.grad, rtol=1e-10, atol=1e-12)


def test_scan_gradient_is_the_slope():
    t, cu, rand = _case((7,), 2, seed=1)
    h0, dfin, dout = rand(1, 2), rand(1, 2), rand(7, 2)
    got = R.scan_bwd(t, cu, dout, h0, dfin)
    for name, key in (("dr", "r"), ("dA", "A"), ("dx", "x")):
        d = torch.randn(t[key].shape, generator=torch.Generator().manual_seed(3), dtype=f64)
        up, down = dict(t), dict(t)
        up[key], down[key] = t[key] + 1e-6 * d, t[key] - 1e-6 * d
        slope = (_loss(up, cu, h0, dout, dfin) - _loss(down, cu, h0, dout, dfin)) / 2e-6
        assert abs(slope - (got[name][0] * d).sum()) < 1e-7 * (1 + abs(slope)), name


def test_norm_gradients_are_the_formulas():
    g = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, dtype=f64)  # noqa: E731
    x, z, w, dy, ds = rand(4, 12), rand(4, 12), rand(12), rand(4, 12), rand(4, 12)
    for gate in (False, True):
        leaves = [v.clone().requires_grad_() for v in (x, z, w)]
        v = leaves[0] * leaves[1] * torch.sigmoid(leaves[1]) if gate else leaves[0]
        by = v.view(4, 3, 4)
        y = (by / torch.sqrt((by * by).mean(-1, keepdim=True) + 1e-5)).view(4, 12) * leaves[2]
        ((y * dy).sum() + (0 if gate else (leaves[0] * ds).sum())).backward()
        got = R.norm_bwd(x, w, dy, z=z if gate else None, ds=None if gate else ds, group=4)
        assert torch.allclose(got["dx"][0], leaves[0].grad, rtol=1e-10, atol=1e-12)
        assert torch.allclose(got["dweight"][0], leaves[2].grad, rtol=1e-10, atol=1e-12)
        if gate:
            assert torch.allclose(got["dz"][0], leaves[1].grad, rtol=1e-10, atol=1e-12)
        assert torch.allclose(R.norm(x, w, z=z if gate else None, group=4)[0], y.detach(), rtol=1e-12, atol=1e-14)
