"""The references that the packed-token operators are tested against, held to
differences of the loss, and the 8-bit states' definition."""
import pytest
import torch

from tests import varlen_ref as R


def _case(seed=0, lens=(5, 0, 70), h=2, G=1, n=4):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    t = dict(x=torch.randn(T, h, R.P, generator=g, dtype=R.f64), dt=torch.randn(T, h, generator=g, dtype=R.f64) - 2,
             A=-1 - torch.rand(h, generator=g, dtype=R.f64), B=torch.randn(T, G, n, generator=g, dtype=R.f64),
             C=torch.randn(T, G, n, generator=g, dtype=R.f64), D=torch.randn(h, generator=g, dtype=R.f64),
             dt_bias=0.1 * torch.randn(h, generator=g, dtype=R.f64), softplus=True)
    return t, R.sequences(lens), torch.randn(T, h, R.P, generator=g, dtype=R.f64)


def _shifted_loss(t, cu, dout, shift):
    """sum(dout out) of the recurrence with a constant added to every chunk's
    entering state (what the 8 bits change), and 0.5 of the last states' sum."""
    total = 0.0
    for s in range(len(cu) - 1):
        S = None
        for c in range(-(-(cu[s + 1] - cu[s]) // R.Q)):
            lo, hi = cu[s] + c * R.Q, min(cu[s + 1], cu[s] + (c + 1) * R.Q)
            e = R.entry(cu, s, c)
            S = shift[e] if S is None else S + shift[e]
            part = {k: (v[lo:hi] if k in ("x", "dt", "B", "C") else v) for k, v in t.items()}
            out, _, last, _, _ = R.scan_fwd(part, [0, hi - lo], S[None])
            total = total + (out * dout[lo:hi]).sum()
            S = last[0]
        if S is not None:
            total = total + 0.5 * S.sum()
    return total


def test_scan_gradients_are_the_loss_differences():
    t, cu, dout = _case()
    _, _, _, _, held = R.scan_fwd(t, cu)
    slots = cu[-1] // R.Q + len(cu) - 1
    codes = torch.zeros(slots, 2, R.P, 4, dtype=torch.int8)
    scales = torch.ones(slots, 2, R.P)
    shift = {}
    # the entering states as the 8-bit restarts change them
    S = {}
    for s in range(len(cu) - 1):
        S = None
        for c in range(-(-(cu[s + 1] - cu[s]) // R.Q)):
            e = R.entry(cu, s, c)
            S = torch.zeros(2, R.P, 4, dtype=R.f64) if S is None else S
            codes[e], scales[e] = R.to_8_bits(held[e][0].float())
            q = codes[e].to(R.f64) * scales[e].to(R.f64)[..., None]
            shift[e] = q - S
            lo, hi = cu[s] + c * R.Q, min(cu[s + 1], cu[s] + (c + 1) * R.Q)
            part = {k: (v[lo:hi] if k in ("x", "dt", "B", "C") else v) for k, v in t.items()}
            S = R.scan_fwd(part, [0, hi - lo], q[None])[2][0]
    grads = R.scan_bwd(t, cu, dout, codes, scales, torch.full((3, 2, R.P, 4), 0.5, dtype=R.f64))
    g = torch.Generator().manual_seed(5)
    for name, key in (("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dA", "A"), ("dD", "D"), ("ddt_bias", "dt_bias")):
        way = torch.randn(t[key].shape, generator=g, dtype=R.f64)
        h = 1e-5
        up = _shifted_loss({**t, key: t[key] + h * way}, cu, dout, shift)
        down = _shifted_loss({**t, key: t[key] - h * way}, cu, dout, shift)
        want = (grads[name][0] * way).sum()
        assert abs((up - down) / (2 * h) - want) <= 1e-6 * (1 + abs(want)), name


def test_conv_gradients_are_the_loss_differences():
    g = torch.Generator().manual_seed(1)
    cu, C = R.sequences([1, 0, 2, 9]), 5
    x, dout = torch.randn(12, C, generator=g, dtype=R.f64), torch.randn(12, C, generator=g, dtype=R.f64)
    w, b = torch.randn(C, 4, generator=g, dtype=R.f64), torch.randn(C, generator=g, dtype=R.f64)
    grads = R.conv_bwd(x, w, b, cu, dout, True)
    for name, k in (("dx", 0), ("dweight", 1), ("dbias", 2)):
        args = [x, w, b]
        way = torch.randn(args[k].shape, generator=g, dtype=R.f64)
        side = []
        for sign in (1, -1):
            moved = list(args)
            moved[k] = args[k] + sign * 1e-6 * way
            side.append((R.conv_fwd(*moved, cu, True)[0] * dout).sum())
        want = (grads[name][0] * way).sum()
        assert abs((side[0] - side[1]) / 2e-6 - want) <= 1e-6 * (1 + abs(want)), name


@pytest.mark.parametrize("top,scale", [(127.0, 1.0), (127.0001, 2.0), (63.5, 0.5), (1.0, 2.0 ** -6), (0.0, 2.0 ** -100)])
def test_8_bit_scale(top, scale):
    codes, s = R.to_8_bits(torch.tensor([[top, -0.3 * top, 0.0]]))
    assert s.item() == scale
    assert (codes.double() * s.double()[..., None] - torch.tensor([top, -0.3 * top, 0.0])).abs().max() <= scale / 2
    assert codes.abs().max() <= 127
