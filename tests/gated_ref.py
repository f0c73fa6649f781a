"""Plain 64-bit references of a gated recurrent block's operators (recurrence,
gradient, step, norm and its gradient) on the CPU, each result with a bound on
what fp32 arithmetic may put beside it.

The bounds are carried along with the values.  With u = 2^-24, the largest
relative error of one fp32 rounding, the hardware exp2, reciprocal and inverse
square root are within one ulp, 2 u:
  sigma(v): the gate's sum with its bias |v| u, the product with log2 e and that
    constant 2 |v| u in the exponent, exp2, the sum and the reciprocal 5 u
  a = exp(y), y = A rho: |y| times rho's and the product's error, exp2 2 u
  m = sqrt(1 - a^2): half of its square's error, which has y's and six roundings
  a product of k factors adds k - 1 roundings.
The recurrence's bound goes through the recurrence itself: a step multiplies
what is off by a, and adds a's error times the magnitude it acts on, the
input's error and three roundings (a step's own, and what a token pays for the
products and sums in which tiles are joined); 64 u of the magnitude stand for
the joining of a few tiles where a sequence is short.  Sums over tokens are
taken in fp32 over at most 128 terms, then in 64 bits.

A result in 16 bits is off by its rounding too, half a step, finfo(io).eps / 2
of its value.
"""
import torch

U = 2.0 ** -24
JOIN = 64
f64 = torch.float64


def half_step(dtype):
    return 0.0 if dtype in (f64, torch.float32) else torch.finfo(dtype).eps / 2


def close(got, ref, err, io, what):
    """|got - ref| <= half a step of io + err, element by element."""
    got = got.detach().cpu().to(f64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = half_step(io) * (ref.abs() + err) + err
    if io == torch.float16:
        tol = tol + 2.0 ** -25   # half of its smallest step
    worst = ((got - ref).abs() - tol).max().item() if ref.numel() else -1.0
    assert worst <= 0.0, f"{what}: over the bound by {worst:.3e} (largest error {(got - ref).abs().max():.3e})"


def sequences(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def token(x, r, i, A, rb, ib):
    """What a token makes of its inputs, and the relative errors of it."""
    vr, vi = r.to(f64), i.to(f64)
    vr = vr if rb is None else vr + rb.to(f64)
    vi = vi if ib is None else vi + ib.to(f64)
    rho, iota = torch.sigmoid(vr), torch.sigmoid(vi)
    y = A.to(f64) * rho
    a = torch.exp(y)
    m = torch.sqrt((-torch.expm1(2 * y)).clamp(min=0))
    e_rho, e_iota = U * (3 * vr.abs() + 5), U * (3 * vi.abs() + 5)
    e_a = y.abs() * (e_rho + 3 * U) + 2 * U
    e_m = 0.5 * (e_rho + e_a) * (1 + y.abs()) + 6 * U
    return dict(x=x.to(f64), rho=rho, iota=iota, a=a, m=m, e_rho=e_rho, e_iota=e_iota, e_a=e_a, e_m=e_m)


def scan(t, cu, h0=None):
    """States after and before every token and their bounds (rows of tokens of
    no sequence 0), and the last states; t: x, r, i, A, r_bias, i_bias."""
    T, C = t["x"].shape
    g = token(t["x"], t["r"], t["i"], t["A"], t.get("r_bias"), t.get("i_bias"))
    after, before, err, err_before, mag, mag_before = (torch.zeros(T, C, dtype=f64) for _ in range(6))
    last = torch.zeros(len(cu) - 1, C, dtype=f64) if h0 is None else h0.to(f64).clone()
    last_err = torch.zeros_like(last)
    for s in range(len(cu) - 1):
        h, e = last[s].clone(), torch.zeros(C, dtype=f64)
        n = h.abs()
        for k in range(cu[s], cu[s + 1]):
            before[k], err_before[k], mag_before[k] = h, e + JOIN * U * n, n
            a, b = g["a"][k], g["m"][k] * g["iota"][k] * g["x"][k]
            e_b = g["e_m"][k] + g["e_iota"][k] + 3 * U
            e = a * e + a * g["e_a"][k] * n + e_b * b.abs()
            h, n = a * h + b, a * n + b.abs()
            e = e + 3 * U * n
            after[k], err[k], mag[k] = h, e + JOIN * U * n, n
        if cu[s + 1] > cu[s]:
            last[s], last_err[s] = h, err[cu[s + 1] - 1]
    return dict(after=after, err=err, before=before, err_before=err_before, mag_before=mag_before, last=last, last_err=last_err,
                gates=g)


def scan_cached(t, cu, state, seen, slots):
    """The forward from and to a cache: the outputs, and the cache afterwards,
    each with its bound."""
    C = t["x"].shape[1]
    h0 = torch.zeros(len(cu) - 1, C, dtype=f64)
    for s in range(len(cu) - 1):
        if 0 <= slots[s] < state.shape[0] and seen[s] > 0:
            h0[s] = state[slots[s]].to(f64)
    r = scan(t, cu, h0)
    cache, err = state.to(f64).clone(), torch.zeros(state.shape, dtype=f64)
    for s in range(len(cu) - 1):
        if 0 <= slots[s] < state.shape[0] and cu[s + 1] > cu[s]:
            cache[slots[s]], err[slots[s]] = r["last"][s], r["last_err"][s]
    return r["after"], r["err"], cache, err


def scan_bwd(t, cu, dout, h0=None, dfinal=None):
    """{name: (gradient, bound)}."""
    T, C = t["x"].shape
    f = scan(t, cu, h0)
    g = f["gates"]
    A = t["A"].to(f64)
    adj, e_adj, mag = (torch.zeros(T, C, dtype=f64) for _ in range(3))
    live = torch.zeros(T, 1, dtype=f64)
    dinit = torch.zeros(len(cu) - 1, C, dtype=f64) if dfinal is None else dfinal.to(f64).clone()
    e_init = torch.zeros_like(dinit)
    for s in range(len(cu) - 1):
        come, e, n = dinit[s].clone(), torch.zeros(C, dtype=f64), dinit[s].abs()
        for k in range(cu[s + 1] - 1, cu[s] - 1, -1):
            live[k] = 1
            G, n = dout[k].to(f64) + come, dout[k].to(f64).abs() + n
            e = e + 3 * U * n
            adj[k], e_adj[k], mag[k] = G, e + JOIN * U * n, n
            a = g["a"][k]
            e = a * e + a * g["e_a"][k] * n
            come, n = a * G, a * n
        dinit[s], e_init[s] = come, e + JOIN * U * n
    over_m = torch.where(g["m"] > 0, 1 / g["m"].clamp(min=1e-300), torch.zeros(())) * live
    gated = g["iota"] * g["x"]
    ra = g["rho"] * g["a"]
    inner = f["before"] - g["a"] * over_m * gated
    inner_mag = f["mag_before"] + g["a"] * over_m * gated.abs()
    e_inner = f["err_before"] + (g["e_a"] + g["e_m"] + g["e_iota"] + 4 * U) * g["a"] * over_m * gated.abs() + U * inner_mag
    q = adj * ra * inner
    q_mag = mag * ra * inner_mag
    e_q = e_adj * ra * inner_mag + mag * ra * e_inner + (g["e_rho"] + g["e_a"] + 4 * U) * q_mag
    # 1 - sigma is off by sigma's error
    left, e_left = 1 - g["rho"], g["e_rho"] * g["rho"] + U
    dr = A * left * q
    e_dr = A.abs() * (left * e_q + e_left * q_mag + 3 * U * left * q_mag)
    dx = adj * g["m"] * g["iota"]
    e_dx = e_adj * g["m"] * g["iota"] + (g["e_m"] + g["e_iota"] + 3 * U) * mag * g["m"] * g["iota"]
    closed, e_closed = 1 - g["iota"], g["e_iota"] * g["iota"] + U
    di = adj * g["m"] * gated * closed
    e_di = ((e_adj + (g["e_m"] + g["e_iota"] + 5 * U) * mag) * closed + mag * e_closed) * g["m"] * gated.abs()
    r = {"dx": (dx * live, e_dx * live), "dr": (dr * live, e_dr * live), "di": (di * live, e_di * live)}
    for name, v, e in (("dA", q, e_q), ("dr_bias", dr, e_dr), ("di_bias", di, e_di)):
        v, e = v * live, e * live
        r[name] = (v.sum(0), e.sum(0) + 130 * U * v.abs().sum(0))
    r["dinitial_states"] = (dinit, e_init)
    return r


# ---- norm -------------------------------------------------------------------

def _groups(v, n):
    return v.view(v.shape[0], -1, n)


def normed(x, residual, z):
    """What is normalised, its relative error, and what the stream then holds."""
    if residual is not None:
        held = (x.float() + residual.float()).to(residual.dtype)
        return held.to(f64), torch.zeros(()), held
    if z is not None:
        zf = z.to(f64)
        return x.to(f64) * zf * torch.sigmoid(zf), U * (3 * zf.abs() + 8), None
    return x.to(f64), torch.zeros(()), None


# A lane adds at most 64 squares and 8 more partial sums join: 72 u of a sum of
# squares, half of that in its root; mean, eps, reciprocal and root 8 u.
ROOT = 44


def norm(x, weight, residual=None, z=None, group=None, eps=1e-5):
    """(y, bound, residual_out)."""
    v, e_v, held = normed(x, residual, z)
    n = group or x.shape[1]
    by = _groups(v, n)
    rstd = 1 / torch.sqrt((by * by).mean(-1, keepdim=True) + eps)
    e_sum = e_v if e_v.dim() == 0 else _groups(e_v.expand_as(v), n).amax(-1, keepdim=True).expand_as(by).reshape(v.shape)
    y = (by * rstd).view_as(v) * weight.to(f64)
    return y, y.abs() * (e_v + e_sum + (ROOT + 3) * U), held


def norm_bwd(x, weight, dy, z=None, ds=None, group=None, eps=1e-5):
    """{name: (gradient, bound)}; x: what was normalised, before the gate."""
    n = group or x.shape[1]
    v, e_v, _ = normed(x, None, z)
    e_v = e_v.expand_as(v)
    xf, w, g = x.to(f64), weight.to(f64), dy.to(f64) * weight.to(f64)
    by, gb, eb = _groups(v, n), _groups(g, n), _groups(e_v, n)
    e_top = eb.amax(-1, keepdim=True)
    rstd = 1 / torch.sqrt((by * by).mean(-1, keepdim=True) + eps)
    hat = by * rstd
    dot, dot_mag = (gb * hat).mean(-1, keepdim=True), (gb * hat).abs().mean(-1, keepdim=True)
    dv = rstd * (gb - hat * dot)
    mag = rstd * (gb.abs() + hat.abs() * dot_mag)
    # the dot product's own sum: 72 u; hat's twice, its and the root's error
    e_dv = (mag * (4 * e_top + (72 + 3 * ROOT + 10) * U)).view_as(v)
    dv, mag = dv.view_as(v), mag.view_as(v)
    hat = hat.view_as(v)
    e_hat = hat.abs() * (e_v + e_top.expand_as(by).reshape(v.shape) + (ROOT + 2) * U)
    terms = dy.to(f64) * hat
    # a lane adds a column's rows one after another in fp32, at most 256 of them, then in 64 bits
    r = {"dweight": (terms.sum(0), (dy.to(f64).abs() * e_hat).sum(0) + 260 * U * terms.abs().sum(0))}
    if z is None:
        dx, e_dx = dv, e_dv
        if ds is not None:
            dx = dx + ds.to(f64)
            e_dx = e_dx + U * (mag + ds.to(f64).abs())
    else:
        zf = z.to(f64)
        sg = torch.sigmoid(zf)
        silu, slope = zf * sg, sg * (1 + zf * (1 - sg))
        e_silu = U * (3 * zf.abs() + 8)
        dx, e_dx = dv * silu, e_dv * silu.abs() + mag * silu.abs() * e_silu
        e_slope = e_silu * sg * (1 + 2 * zf.abs())
        r["dz"] = (dv * xf * slope, xf.abs() * (e_dv * slope.abs() + mag * e_slope + 3 * U * mag * slope.abs()))
    r["dx"] = r["dresidual"] = (dx, e_dx)
    return r


def e4m3_step(y, scale):
    """Half a step of e4m3 at y, for codes that stand for code * scale: three
    fraction bits, the smallest step 2^-9."""
    return torch.maximum(y.abs() * 2.0 ** -4, scale * 2.0 ** -10)
