"""Plain 64-bit references of the packed-token operators (the Mamba-2 mixer's
conv, scan and step), token by token, on the CPU, with the sum of the terms'
magnitudes beside every result.

Tolerances.  A result in io type is off by its rounding, half a step,
finfo(io).eps / 2 of its value.  Before that rounding the kernels work in
fp32: a derived matrix operand is a bf16 head and tail (its residual is below
2^-17 of it, at most three such factors in a term), exp(cs) takes the rounding
of cs (|cs| * 2^-23, |cs| < 64 here: 2^-17), the hardware exp2, log2 and
reciprocal give 2^-22, and a sum of up to 512 terms in fp32 adds 2^-24 of the
partial sums for each.  Together below 2^-14 of the sum of the magnitudes,
which is what FP32 allows.  The convolution and the step use no matrix
operand: 2^-19 covers their ten roundings and two hardware functions.
"""
import math

import torch

P, Q, W = 64, 64, 4
FP32 = 2.0 ** -14
SHORT = 2.0 ** -19
f64 = torch.float64


def half_step(dtype):
    return 0.0 if dtype == f64 else torch.finfo(dtype).eps / 2


def close(got, ref, mag, io, what, fp32=FP32):
    """|got - ref| <= half a step of io + fp32 * magnitude, element by element
    (fp16's smallest step, 2^-25, below its normal numbers)."""
    got = got.detach().cpu().to(f64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = half_step(io) * (ref.abs() + fp32 * mag) + fp32 * mag
    if io == torch.float16:
        tol = tol + 2.0 ** -25
    worst = ((got - ref).abs() - tol).max().item() if ref.numel() else -1.0
    assert worst <= 0.0, f"{what}: over the bound by {worst:.3e} (largest error {(got - ref).abs().max():.3e})"


def sequences(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# ---- convolution ----------------------------------------------------------

def conv_inputs(x, cu, ring, seen, slots):
    """(T, 4, C) float64: what every token's output sees."""
    v = torch.zeros(x.shape[0], W, x.shape[1], dtype=f64)
    for s in range(len(cu) - 1):
        for t in range(cu[s], cu[s + 1]):
            for k in range(W):
                pos = t - cu[s] - (W - 1) + k
                if pos >= 0:
                    v[t, k] = x[cu[s] + pos].to(f64)
                elif ring is not None and seen is not None and seen[s] + pos >= 0 and 0 <= slots[s] < ring.shape[0]:
                    v[t, k] = ring[slots[s], :, (seen[s] + pos) % ring.shape[2]].to(f64)
    return v


def silu(v):
    return v / (1.0 + torch.exp(-v))


def conv_fwd(x, w, bias, cu, act, ring=None, seen=None, slots=None):
    """(out, magnitude, ring after)"""
    n = len(cu) - 1
    slots = list(range(n)) if slots is None else slots
    v = conv_inputs(x, cu, ring, seen, slots)
    b = torch.zeros(x.shape[1], dtype=f64) if bias is None else bias.to(f64)
    pre = (v * w.to(f64).t()).sum(1) + b
    mag = (v.abs() * w.to(f64).abs().t()).sum(1) + b.abs()
    after = None
    if ring is not None:
        after = ring.clone()
        for s in range(n):
            if not 0 <= slots[s] < ring.shape[0]:
                continue
            first = 0 if seen is None else seen[s]
            for t in range(max(cu[s], cu[s + 1] - ring.shape[2]), cu[s + 1]):
                after[slots[s], :, (first + t - cu[s]) % ring.shape[2]] = x[t]
    # silu's slope is at most 1.1
    return (silu(pre) if act else pre), 1.1 * mag, after


def conv_bwd(x, w, bias, cu, dout, act):
    """{name: (gradient, magnitude)}"""
    v = conv_inputs(x, cu, None, None, [0] * len(cu))
    w, g = w.to(f64), dout.to(f64)
    b = torch.zeros(x.shape[1], dtype=f64) if bias is None else bias.to(f64)
    pre = (v * w.t()).sum(1) + b
    pre_mag = (v.abs() * w.abs().t()).sum(1) + b.abs()
    sg = 1.0 / (1.0 + torch.exp(-pre))
    da = g * (sg + pre * sg * (1 - sg)) if act else g
    # silu' is at most 1.1 and its slope at most 1/2
    mag = g.abs() * (1.1 + 0.5 * pre_mag) if act else g.abs()
    dx, dxm = torch.zeros_like(g), torch.zeros_like(g)
    for s in range(len(cu) - 1):
        for t in range(cu[s], cu[s + 1]):
            for k in range(W):
                src = t - (W - 1) + k
                if src >= cu[s]:
                    dx[src] += w[:, k] * da[t]
                    dxm[src] += w[:, k].abs() * mag[t]
    return {"dx": (dx, dxm), "dweight": ((da[:, None] * v).sum(0).t(), (mag[:, None] * v.abs()).sum(0).t()),
            "dbias": (da.sum(0), mag.sum(0))}


# ---- scan -----------------------------------------------------------------

def softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)


def steps(dt, dt_bias, use_softplus, limit):
    """(dt', d dt' / d dt)"""
    v = dt.to(f64) + (0 if dt_bias is None else dt_bias.to(f64))
    d = softplus(v) if use_softplus else v
    slope = 1.0 / (1.0 + torch.exp(-v)) if use_softplus else torch.ones_like(v)
    if limit is not None:
        slope = slope * ((d >= limit[0]) & (d <= limit[1]))
        d = d.clamp(limit[0], limit[1])
    return d, slope


def to_8_bits(state):
    """(codes, scales) of a float32 state (..., n), by the definition."""
    top = state.abs().amax(-1).to(f64)
    scale = torch.exp2(torch.ceil(torch.log2((top / 127.0).clamp(min=2.0 ** -100))))
    scale = torch.where(torch.isfinite(top), scale, torch.full_like(scale, math.nan))
    codes = torch.where(torch.isfinite(scale)[..., None], torch.round(state.to(f64) / scale[..., None]), torch.zeros(1, dtype=f64))
    return codes.nan_to_num(0.0).to(torch.int8), scale.float()


def entry(cu, s, chunk):
    return cu[s] // Q + s + chunk


def scan_fwd(t, cu, first=None):
    """t: dict of x (T,h,p), dt, A, B (T,g,n), C, and D, z, dt_bias, softplus,
    limit.  first: (nseq,h,p,n) or None.  Returns out, its magnitude, the last
    states, their magnitude, and {entry: (entering state, its magnitude)}."""
    x, B, C, A = t["x"].to(f64), t["B"].to(f64), t["C"].to(f64), t["A"].to(f64)
    T, h, _ = x.shape
    rep = h // B.shape[1]
    d, _ = steps(t["dt"], t.get("dt_bias"), t.get("softplus", False), t.get("limit"))
    keep = torch.exp(d * A)
    D = t.get("D")
    D = torch.zeros(h, 1, dtype=f64) if D is None else D.to(f64).reshape(h, -1)
    out, mag = torch.zeros_like(x), torch.zeros_like(x)
    n = B.shape[2]
    last = torch.zeros(len(cu) - 1, h, P, n, dtype=f64)
    lastm = torch.zeros_like(last)
    held = {}
    for s in range(len(cu) - 1):
        S = torch.zeros(h, P, n, dtype=f64) if first is None else first[s].to(f64).clone()
        M = S.abs()
        for i, k in enumerate(range(cu[s], cu[s + 1])):
            if i % Q == 0:
                held[entry(cu, s, i // Q)] = (S.clone(), M.clone())
            b, c = B[k].repeat_interleave(rep, 0), C[k].repeat_interleave(rep, 0)
            add = (d[k][:, None] * x[k])[:, :, None] * b[:, None, :]
            S = keep[k][:, None, None] * S + add
            M = keep[k][:, None, None] * M + add.abs()
            out[k] = (S * c[:, None, :]).sum(-1) + D * x[k]
            mag[k] = (M * c.abs()[:, None, :]).sum(-1) + (D * x[k]).abs()
        last[s], lastm[s] = S, M
    z = t.get("z")
    if z is not None:
        gate = silu(z.to(f64))
        out, mag = out * gate, mag * gate.abs()
    return out, mag, last, lastm, held


def scan_bwd(t, cu, dout, codes, scales, dlast=None):
    """{name: (gradient, magnitude)} from the recurrence's adjoint, every chunk
    re-run from its 8-bit state."""
    x, B, C, A, g = t["x"].to(f64), t["B"].to(f64), t["C"].to(f64), t["A"].to(f64), dout.to(f64)
    T, h, _ = x.shape
    G, n = B.shape[1], B.shape[2]
    rep = h // G
    d, slope = steps(t["dt"], t.get("dt_bias"), t.get("softplus", False), t.get("limit"))
    keep = torch.exp(d * A)
    D = t.get("D")
    Df = torch.zeros(h, 1, dtype=f64) if D is None else D.to(f64).reshape(h, -1)
    z = {k: [torch.zeros_like(v), torch.zeros_like(v)] for k, v in
         dict(dx=x, dB=B, dC=C, ddt=d, dinitial_states=torch.zeros(len(cu) - 1, h, P, n, dtype=f64)).items()}
    dA, dAm, db, dbm = (torch.zeros(h, dtype=f64) for _ in range(4))
    up = lambda v: v.repeat_interleave(rep, 0)  # noqa: E731
    down = lambda v: v.reshape(G, rep, n).sum(1)  # noqa: E731
    for s in range(len(cu) - 1):
        lo, hi = cu[s], cu[s + 1]
        adj = torch.zeros(h, P, n, dtype=f64) if dlast is None else dlast[s].to(f64).clone()
        adjm = adj.abs()
        for c in range((hi - lo - 1) // Q, -1, -1):
            S = codes[entry(cu, s, c)].to(f64) * scales[entry(cu, s, c)].to(f64)[..., None]
            M = S.abs()
            ks = range(lo + c * Q, min(hi, lo + (c + 1) * Q))
            past = []
            path = torch.zeros(h, dtype=f64)   # what the chunk's running sums add up
            for k in ks:
                past.append((S, M))
                add = (d[k][:, None] * x[k])[:, :, None] * up(B[k])[:, None, :]
                S, M = keep[k][:, None, None] * S + add, keep[k][:, None, None] * M + add.abs()
                path += (g[k].abs()[:, :, None] * M * up(C[k]).abs()[:, None, :]).sum((1, 2))
                z["dC"][0][k] = down(torch.einsum("hp,hpn->hn", g[k], S))
                z["dC"][1][k] = down(torch.einsum("hp,hpn->hn", g[k].abs(), M))
            path += (adjm * M).sum((1, 2))
            tail = []
            for k in reversed(ks):
                add = g[k][:, :, None] * up(C[k])[:, None, :]
                adj, adjm = adj + add, adjm + add.abs()
                S, M = past[k - ks[0]]
                ab, abm = (adj * up(B[k])[:, None, :]).sum(-1), (adjm * up(B[k]).abs()[:, None, :]).sum(-1)
                z["dx"][0][k] = d[k][:, None] * ab + Df * g[k]
                z["dx"][1][k] = d[k].abs()[:, None] * abm + (Df * g[k]).abs()
                z["dB"][0][k] = down(d[k][:, None] * torch.einsum("hp,hpn->hn", x[k], adj))
                z["dB"][1][k] = down(d[k].abs()[:, None] * torch.einsum("hp,hpn->hn", x[k].abs(), adjm))
                direct, directm = (ab * x[k]).sum(-1), (abm * x[k].abs()).sum(-1)
                through = keep[k] * (adj * S).sum((1, 2))
                path += d[k].abs() * directm
                z["ddt"][0][k] = (direct + A * through) * slope[k]
                tail.append((k, directm))
                dA += d[k] * through
                db += z["ddt"][0][k]
                adj, adjm = keep[k][:, None, None] * adj, keep[k][:, None, None] * adjm
            for k, directm in tail:
                z["ddt"][1][k] = (directm + A.abs() * path) * slope[k]
                dAm += d[k].abs() * path
                dbm += z["ddt"][1][k]
        z["dinitial_states"][0][s], z["dinitial_states"][1][s] = adj, adjm
    r = {k: tuple(v) for k, v in z.items()}
    r["dA"], r["ddt_bias"] = (dA, dAm), (db, dbm)
    gx = g * x
    if D is not None:
        r["dD"] = (gx.sum(0), gx.abs().sum(0)) if D.dim() == 2 else (gx.sum((0, 2)), gx.abs().sum((0, 2)))
    return r
