"""The packed-token operators on the GPU against the 64-bit references of
varlen_ref.py (whose head derives the tolerances)."""
import pytest
import torch

from state_space_model_scan_amd import binding
from tests import varlen_ref as R
from tests.harness import log

pytestmark = pytest.mark.gpu
bf, f16, f32, i32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, dtype=f32, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _dev(v):
    return v.cuda() if isinstance(v, torch.Tensor) else v


def _ints(v):
    return torch.tensor(v, dtype=i32, device="cuda")


# ---- convolution ----------------------------------------------------------

LENS = [(1,), (5,), (3, 0, 1, 2, 40, 0), (64, 65), (16, 16, 200), (0, 0, 7)]


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("channels", [8, 40, 67, 1032])
@pytest.mark.parametrize("lens", LENS)
def test_conv_fwd(io, channels, lens):
    log(f"[conv fwd] {io} channels={channels} lens={lens}")
    g = _gen(channels + sum(lens))
    cu = R.sequences(lens)
    x, w, b = _randn(g, cu[-1], channels, dtype=io), _randn(g, channels, 4, scale=0.5), _randn(g, channels)
    ref, mag, _ = R.conv_fwd(x, w, b, cu, True)
    out = binding.causal_conv1d_varlen_fwd(x.cuda(), w.cuda(), _ints(cu), bias=b.cuda(), activation="silu")
    R.close(out, ref, mag, io, "out", R.SHORT)
    ref, mag, _ = R.conv_fwd(x, w, None, cu, False)
    out = binding.causal_conv1d_varlen_fwd(x.cuda(), w.cuda(), _ints(cu))
    R.close(out, ref, mag, io, "out without bias and activation", R.SHORT)


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("ring_len", [4, 7])
def test_conv_fwd_cache(io, ring_len):
    lens, channels = (5, 1, 0, 2, 30, 3, 9), 72
    seen, slots = [0, 1, 2, 3, 4, 1000, 2], [6, 2, 0, 7, 1, -1, 99]
    log(f"[conv cache] {io} ring={ring_len}")
    g, cu = _gen(ring_len), R.sequences(lens)
    x, w, b = _randn(g, cu[-1], channels, dtype=io), _randn(g, channels, 4, scale=0.5), _randn(g, channels)
    ring = _randn(g, 8, channels, ring_len, dtype=io)
    ring[2, :, 1:] = float("nan")   # entries of positions that do not exist yet are never looked at
    ref, mag, after = R.conv_fwd(x, w, b, cu, True, ring, seen, slots)
    dring = ring.cuda()
    # a part of wider rows, and outputs into a part of wider rows
    wide = torch.full((cu[-1], channels + 24), float("nan"), dtype=io, device="cuda")
    wide[:, 16:16 + channels] = x.cuda()
    room = torch.zeros(cu[-1], channels + 8, dtype=io, device="cuda")
    out = binding.causal_conv1d_varlen_fwd(wide[:, 16:16 + channels], w.cuda(), _ints(cu), bias=b.cuda(), activation="silu",
                                           conv_state=dring, cache_seqlens=_ints(seen), slots=_ints(slots),
                                           out=room[:, 8:])
    R.close(out, ref, mag, io, "out", R.SHORT)
    assert torch.equal(dring.cpu().view(torch.uint8), after.view(torch.uint8)), "ring"
    assert not room[:, :8].any()


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("channels", [8, 67, 520])
@pytest.mark.parametrize("lens", LENS + [(300, 1, 130)])
def test_conv_bwd(io, channels, lens):
    log(f"[conv bwd] {io} channels={channels} lens={lens}")
    g, cu = _gen(channels + sum(lens)), R.sequences(lens)
    x, w, b = _randn(g, cu[-1], channels, dtype=io), _randn(g, channels, 4, scale=0.5), _randn(g, channels)
    dout = _randn(g, cu[-1], channels, dtype=io)
    for act, bias in (("silu", b), (None, None)):
        ref = R.conv_bwd(x, w, bias, cu, dout, act is not None)
        got = binding.causal_conv1d_varlen_bwd(x.cuda(), w.cuda(), _ints(cu), dout.cuda(),
                                               bias=None if bias is None else bias.cuda(), activation=act)
        R.close(got["dx"], *ref["dx"], io, "dx", R.SHORT)
        R.close(got["dweight"], *ref["dweight"], f32, "dweight", R.SHORT)
        if bias is not None:
            R.close(got["dbias"], *ref["dbias"], f32, "dbias", R.SHORT)


@pytest.mark.parametrize("io,channels", [(bf, 4096), (f32, 1003)])
def test_conv_of_many_tokens(io, channels):
    """As many tokens and channels as the longer runs are taken for, from and to
    a ring; sequences that end inside a run, and ones shorter than it."""
    lens = (3000, 1, 0, 701, 2, 899)
    log(f"[conv many] {io} channels={channels}")
    g, cu = _gen(channels), R.sequences(lens)
    x, w, b = _randn(g, cu[-1], channels, dtype=io), _randn(g, channels, 4, scale=0.5), _randn(g, channels)
    dout, ring, seen = _randn(g, cu[-1], channels, dtype=io), _randn(g, 6, channels, 5, dtype=io), [0, 7, 1, 2, 0, 3]
    ref, mag, after = R.conv_fwd(x, w, b, cu, True, ring, seen, list(range(6)))
    dring = ring.cuda()
    out = binding.causal_conv1d_varlen_fwd(x.cuda(), w.cuda(), _ints(cu), bias=b.cuda(), activation="silu", conv_state=dring,
                                           cache_seqlens=_ints(seen))
    R.close(out, ref, mag, io, "out", R.SHORT)
    assert torch.equal(dring.cpu().view(torch.uint8), after.view(torch.uint8)), "ring"
    ref = R.conv_bwd(x, w, b, cu, dout, True)
    got = binding.causal_conv1d_varlen_bwd(x.cuda(), w.cuda(), _ints(cu), dout.cuda(), bias=b.cuda(), activation="silu")
    R.close(got["dx"], *ref["dx"], io, "dx", R.SHORT)
    for k in ("dweight", "dbias"):   # 32 tokens in a row in 32 bits, four such runs, some 8 roundings of a term: below 2^-18
        R.close(got[k], *ref[k], f32, k, 2 * R.SHORT)


def test_conv_keeps_to_its_sequence():
    """Infinities and NaN of one sequence reach no other, forward or backward."""
    cu = [0, 4, 9, 15]
    g = _gen(3)
    x, w = _randn(g, 15, 16, dtype=bf), _randn(g, 16, 4)
    x[4:9] = float("nan")
    dout = _randn(g, 15, 16, dtype=bf)
    out = binding.causal_conv1d_varlen_fwd(x.cuda(), w.cuda(), _ints(cu)).cpu()
    dx = binding.causal_conv1d_varlen_bwd(x.cuda(), w.cuda(), _ints(cu), dout.cuda(), activation="silu")["dx"].cpu()
    for v in (out, dx):
        assert torch.isfinite(v[:4]).all() and torch.isfinite(v[9:]).all() and torch.isnan(v[4:9]).any()


# ---- scan -----------------------------------------------------------------

def _scan_case(seed, lens, h, G, n, z=False, D="head", bias=True, softplus=True, limit=None):
    g, T = _gen(seed), sum(lens)
    t = dict(x=_randn(g, T, h, R.P, dtype=bf), A=-1 - 7 * torch.rand(h, generator=g),
             B=_randn(g, T, G, n, dtype=bf), C=_randn(g, T, G, n, dtype=bf),
             D=None if D is None else _randn(g, h) if D == "head" else _randn(g, h, R.P),
             z=_randn(g, T, h, R.P, dtype=bf) if z else None, dt_bias=_randn(g, h, scale=0.1) if bias else None,
             softplus=softplus, limit=limit)
    t["dt"] = _randn(g, T, h, dtype=bf, scale=0.5) - 3 if softplus else (0.02 + 0.1 * torch.rand(T, h, generator=g)).to(bf)
    return t, R.sequences(lens)


def _call(t, strided=False):
    """The tensors on the GPU, with strided=True as parts of wider rows."""
    d = {k: _dev(v) for k, v in t.items() if k not in ("softplus", "limit")}
    if strided:
        T, h, _ = t["x"].shape
        G, n = t["B"].shape[1:]
        row = torch.zeros(T, 8 + h * R.P + 2 * G * n + 8, dtype=bf, device="cuda")
        at = 8
        for k, w in (("x", h * R.P), ("B", G * n), ("C", G * n)):
            part = row[:, at:at + w].view(d[k].shape)
            part.copy_(d[k])
            d[k] = part
            at += w
        wide = torch.zeros(T, 2 * h + 1, dtype=bf, device="cuda")
        wide[:, 1:h + 1] = d["dt"]
        d["dt"] = wide[:, 1:h + 1]
    return d, dict(dt_softplus=t["softplus"], dt_limit=t["limit"])


def _check_scan(t, cu, what, first=None, strided=False, segments=0):
    log(f"[scan] {what} x={tuple(t['x'].shape)} B={tuple(t['B'].shape)} cu={cu} segments={segments}")
    T, h, _ = t["x"].shape
    n, nseq = t["B"].shape[2], len(cu) - 1
    ref, mag, last, lastm, held = R.scan_fwd(t, cu, first)
    d, kw = _call(t, strided)
    state = torch.full((nseq + 1, h, R.P, n), float("nan"), device="cuda")
    slots = list(range(nseq, 0, -1))
    seen = [0] * nseq
    if first is not None:
        for s in range(nseq):
            seen[s] = 1 + s
            state[slots[s]] = first[s].cuda()
    entries = binding.ssd_checkpoint_slots(T, nseq)
    codes = torch.full((entries, h, R.P, n), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((entries, h, R.P), -1.0, device="cuda")
    out = binding.ssd_varlen_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), max(b - a for a, b in zip(cu, cu[1:])),
                                 D=d["D"], z=d["z"], dt_bias=d["dt_bias"], ssm_state=state, cache_seqlens=_ints(seen),
                                 slots=_ints(slots), checkpoints=(codes, scales), seq_segments=segments, **kw)
    R.close(out, ref, mag, bf, f"{what}: out")
    R.close(state[slots], last, lastm, f32, f"{what}: state")
    assert torch.isnan(state[0]).all()
    codes, scales = codes.cpu().double(), scales.cpu().double()
    for e in range(entries):
        if e not in held:
            assert (codes[e] == 77).all() and (scales[e] == -1).all(), f"{what}: entry {e} of no chunk was written"
            continue
        S, M = held[e]
        err = R.FP32 * M.amax(-1)
        assert (torch.frexp(scales[e])[0] == 0.5).all()
        assert ((codes[e] * scales[e][..., None] - S).abs() <= (scales[e] / 2 + err)[..., None]).all(), f"{what}: codes of entry {e}"
        top = S.abs().amax(-1)
        assert (top <= 127 * scales[e] + err).all() and ((scales[e] <= 2.0 ** -100) | (top >= 63.5 * scales[e] - err)).all()


@pytest.mark.parametrize("n", [32, 64, 128])
@pytest.mark.parametrize("lens", [(1,), (63,), (64,), (65,), (3, 0, 1, 130, 64, 0)])
def test_scan_sizes(n, lens):
    t, cu = _scan_case(n + sum(lens), lens, 4, 2, n)
    _check_scan(t, cu, f"n={n}")


@pytest.mark.parametrize("kw", [dict(z=True), dict(D=None, bias=False), dict(D="channel", z=True), dict(softplus=False),
                                dict(limit=(0.03, 0.06)), dict(softplus=False, limit=(0.05, 0.08))])
def test_scan_options(kw):
    t, cu = _scan_case(7, (70, 5), 3, 1, 64, **kw)
    _check_scan(t, cu, str(kw), strided=True)


@pytest.mark.parametrize("segments", [0, 1, 2, 3, 50])
def test_scan_continues_and_splits(segments):
    t, cu = _scan_case(11, (300, 0, 20, 129), 2, 1, 128)
    first = _randn(_gen(2), 4, 2, R.P, 128)
    _check_scan(t, cu, "continued", first=first, segments=segments)


@pytest.mark.parametrize("n", [32, 64, 128])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("D", [None, "head"])
def test_scan_serving(n, z, D):
    """Without 8-bit states: to a cache, and with neither."""
    t, cu = _scan_case(13 * n + z, (130, 0, 1, 64, 70), 3, 1, n, z=z, D=D)
    log(f"[scan serving] n={n} z={z} D={D}")
    ref, mag, last, lastm, _ = R.scan_fwd(t, cu)
    d, kw = _call(t, strided=True)
    args = (d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), 130)
    state = torch.full((5, 3, R.P, n), float("nan"), device="cuda")
    out = binding.ssd_varlen_fwd(*args, D=d["D"], z=d["z"], dt_bias=d["dt_bias"], ssm_state=state, **kw)
    R.close(out, ref, mag, bf, "out")
    full = [0, 2, 3, 4]   # the empty sequence's entry is compared in the test of continued ones
    R.close(state[full], last[full], lastm[full], f32, "state")
    assert torch.equal(binding.ssd_varlen_fwd(*args, D=d["D"], z=d["z"], dt_bias=d["dt_bias"], **kw), out)


def test_scan_without_a_cache_entry():
    """An entry outside the cache: a fresh sequence, nothing written."""
    t, cu = _scan_case(5, (10, 20), 2, 1, 32)
    ref, mag, last, lastm, _ = R.scan_fwd(t, cu)
    d, kw = _call(t)
    state = torch.full((1, 2, R.P, 32), 3.0, device="cuda")
    out = binding.ssd_varlen_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), 20, D=d["D"], dt_bias=d["dt_bias"],
                                 ssm_state=state, cache_seqlens=_ints([5, 5]), slots=_ints([-1, 1]), **kw)
    R.close(out, ref, mag, bf, "out")
    assert (state == 3.0).all()


def test_checkpoints_of_a_row_that_is_not_finite():
    t, cu = _scan_case(5, (130,), 1, 1, 32)
    t["x"][3, 0, 9] = float("inf")
    d, kw = _call(t)
    codes, scales = torch.ones(3, 1, R.P, 32, dtype=torch.int8, device="cuda"), torch.ones(3, 1, R.P, device="cuda")
    binding.ssd_varlen_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), 130, dt_bias=d["dt_bias"],
                           checkpoints=(codes, scales), **kw)
    bad = torch.isnan(scales[1, 0])
    assert bad[9] and bad.sum() == 1 and torch.isfinite(scales[0]).all()


# ---- scan, backward -------------------------------------------------------

def _check_bwd(t, cu, what, dlast=None, strided=False, segments=0):
    log(f"[scan bwd] {what} x={tuple(t['x'].shape)} B={tuple(t['B'].shape)} cu={cu} segments={segments}")
    T, h, _ = t["x"].shape
    G, n = t["B"].shape[1:]
    nseq = len(cu) - 1
    g = _gen(T)
    dout = _randn(g, T, h, R.P, dtype=bf)
    held = R.scan_fwd(t, cu)[4]
    entries = binding.ssd_checkpoint_slots(T, nseq)
    # entries of no chunk hold anything
    codes, scales = torch.full((entries, h, R.P, n), 5, dtype=torch.int8), torch.full((entries, h, R.P), float("nan"))
    for e, (S, _) in held.items():
        codes[e], scales[e] = R.to_8_bits(S.float())
    ref = R.scan_bwd(t, cu, dout, codes, scales, dlast)
    d, kw = _call(t, strided)
    given = {}
    if strided:
        row = torch.full((T, h * R.P + 2 * G * n), float("nan"), dtype=bf, device="cuda")
        given = dict(dx=row[:, :h * R.P].view(T, h, R.P), dB=row[:, h * R.P:h * R.P + G * n].view(T, G, n),
                     dC=row[:, h * R.P + G * n:].view(T, G, n), ddt=torch.zeros(T, h + 3, dtype=bf, device="cuda")[:, 3:])
    held_codes, held_scales = codes.cuda(), scales.cuda()
    if strided:   # laid out head by head
        held_codes = held_codes.transpose(0, 1).contiguous().transpose(0, 1)
        held_scales = held_scales.transpose(0, 1).contiguous().transpose(0, 1)
    call = lambda: binding.ssd_varlen_bwd(  # noqa: E731
        d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), max(b - a for a, b in zip(cu, cu[1:])), dout.cuda(),
        (held_codes, held_scales), D=d["D"], dt_bias=d["dt_bias"], dfinal_states=_dev(dlast),
        want_dinitial_states=True, seq_segments=segments, **given, **kw)
    got = call()
    for k in ("dx", "ddt", "dB", "dC"):
        R.close(got[k], *ref[k], bf, f"{what}: {k}")
    for k in ("dA", "dinitial_states") + (("dD",) if t["D"] is not None else ()) + (("ddt_bias",) if t["dt_bias"] is not None else ()):
        R.close(got[k], *ref[k], f32, f"{what}: {k}")
    first = {k: v.clone() for k, v in got.items()}
    again = call()
    for k, v in first.items():
        assert torch.equal(v, again[k]), f"{what}: {k} differs between two calls"


@pytest.mark.parametrize("n", [32, 64, 128])
@pytest.mark.parametrize("lens", [(1,), (63,), (64,), (65,), (3, 0, 1, 130, 64, 0)])
def test_scan_bwd_sizes(n, lens):
    t, cu = _scan_case(n + sum(lens), lens, 4, 2, n)
    _check_bwd(t, cu, f"n={n}")


@pytest.mark.parametrize("kw", [dict(D=None, bias=False), dict(D="channel"), dict(softplus=False), dict(limit=(0.03, 0.06)),
                                dict(softplus=False, limit=(0.05, 0.08))])
def test_scan_bwd_options(kw):
    t, cu = _scan_case(7, (70, 5), 3, 1, 64, **kw)
    _check_bwd(t, cu, str(kw), strided=True)


@pytest.mark.parametrize("heads,groups", [(1, 1), (19, 1), (6, 3), (34, 2)])
def test_scan_bwd_heads(heads, groups):
    t, cu = _scan_case(heads, (67, 3), heads, groups, 32)
    _check_bwd(t, cu, f"heads={heads} groups={groups}")


@pytest.mark.parametrize("segments", [0, 1, 2, 3, 50])
def test_scan_bwd_segments(segments):
    t, cu = _scan_case(13, (300, 0, 20, 129), 2, 1, 128)
    _check_bwd(t, cu, "segments", dlast=_randn(_gen(4), 4, 2, R.P, 128), segments=segments)


def test_scan_bwd_is_the_forwards():
    """With the checkpoints that the forward wrote: gradients against the
    reference at those codes, and many head blocks (the sum over blocks)."""
    t, cu = _scan_case(3, (200, 77), 40, 1, 128)
    d, kw = _call(t)
    T, h = 277, 40
    codes = torch.zeros(binding.ssd_checkpoint_slots(T, 2), h, R.P, 128, dtype=torch.int8, device="cuda")
    scales = torch.ones(codes.shape[:3], device="cuda")
    args = (d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), 200)
    binding.ssd_varlen_fwd(*args, D=d["D"], dt_bias=d["dt_bias"], checkpoints=(codes, scales), **kw)
    dout = _randn(_gen(9), T, h, R.P, dtype=bf)
    got = binding.ssd_varlen_bwd(*args, dout.cuda(), (codes, scales), D=d["D"], dt_bias=d["dt_bias"], **kw)
    ref = R.scan_bwd(t, cu, dout, codes.cpu(), scales.cpu())
    for k in ("dx", "ddt", "dB", "dC"):
        R.close(got[k], *ref[k], bf, k)
    for k in ("dA", "dD", "ddt_bias"):
        R.close(got[k], *ref[k], f32, k)


# ---- the step -------------------------------------------------------------

def _step_ref(xbc, dt, A, w, ring, state, seen, slots, b, D, z, dt_bias, softplus, limit, G, act):
    batch, h, n = xbc.shape[0], A.shape[0], state.shape[3]
    outs, mags, ring, state, statem = [], [], ring.clone(), state.double().clone(), state.double().abs()
    hp = h * R.P
    for i in range(batch):
        real = 0 <= slots[i] < state.shape[0]
        first = seen[i] if real else 0
        u, um = b.double().clone(), b.double().abs()
        for k in range(4):
            pos = first - 3 + k
            v = xbc[i].double() if k == 3 else ring[slots[i], :, pos % ring.shape[2]].double() if pos >= 0 else None
            if v is not None:
                u, um = u + w[:, k].double() * v, um + (w[:, k].double() * v).abs()
        if real:
            ring[slots[i], :, first % ring.shape[2]] = xbc[i]
        if act:
            u, um = R.silu(u), 1.1 * um
        part = lambda v, a, c: v[a:c].reshape(-1, n).repeat_interleave(h // G, 0)  # noqa: E731
        x, B, C = u[:hp].reshape(h, R.P), part(u, hp, hp + G * n), part(u, hp + G * n, hp + 2 * G * n)
        xm, Bm, Cm = um[:hp].reshape(h, R.P), part(um, hp, hp + G * n), part(um, hp + G * n, hp + 2 * G * n)
        d, _ = R.steps(dt[i], dt_bias, softplus, limit)
        old = state[slots[i]] if first > 0 else torch.zeros(h, R.P, n, dtype=R.f64)
        keep = torch.exp(d * A.double())[:, None, None]
        new = keep * old + (d[:, None] * x)[:, :, None] * B[:, None, :]
        newm = keep * old.abs() + (d.abs()[:, None] * xm)[:, :, None] * Bm[:, None, :]
        Df = D.double().reshape(h, -1)
        y = (new * C[:, None, :]).sum(-1) + Df * x
        ym = (newm * Cm[:, None, :]).sum(-1) + (Df * xm).abs()
        if z is not None:
            gate = R.silu(z[i].double()).reshape(h, R.P)
            y, ym = y * gate, ym * gate.abs()
        if real:
            state[slots[i]], statem[slots[i]] = new, newm
        outs.append(y.reshape(-1))
        mags.append(ym.reshape(-1))
    return torch.stack(outs), torch.stack(mags), ring, state, statem


# the sums over dstate: 128 more roundings of 2^-24
STEP = R.SHORT + 2.0 ** -17


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("n,heads,groups,kw", [
    (32, 3, 1, {}), (64, 4, 2, dict(z=True)), (128, 5, 5, dict(z=True, D="channel", ring=9)),
    (128, 2, 1, dict(limit=(0.03, 0.06))), (64, 2, 2, dict(softplus=False, act=None))])
def test_step(io, n, heads, groups, kw):
    log(f"[step] {io} n={n} heads={heads} groups={groups} {kw}")
    g, batch, hp = _gen(n + heads), 7, heads * R.P
    ch = hp + 2 * groups * n
    seen, slots = [0, 1, 2, 3, 4, 77, 5], [8, 3, 0, 5, 1, -1, 9]
    row = _randn(g, batch, hp + ch + heads, dtype=io)
    softplus, limit, act = kw.get("softplus", True), kw.get("limit"), kw.get("act", "silu")
    if softplus:
        row[:, hp + ch:] -= 3
    else:
        row[:, hp + ch:] = row[:, hp + ch:].abs() * 0.05 + 0.15   # a positive step with the bias
    w, b, A = _randn(g, ch, 4, scale=0.5), _randn(g, ch), -1 - 7 * torch.rand(heads, generator=g)
    D = _randn(g, heads, R.P) if kw.get("D") == "channel" else _randn(g, heads)
    bias = 0.1 * torch.rand(heads, generator=g)
    ring, state = _randn(g, 9, ch, kw.get("ring", 4), dtype=io), _randn(g, 9, heads, R.P, n)
    state[8] = float("nan")    # a new request's entry is not read
    z = row[:, :hp] if kw.get("z") else None
    ref, mag, ring1, state1, statem = _step_ref(row[:, hp:hp + ch], row[:, hp + ch:], A, w, ring, state, seen, slots, b, D, z,
                                                bias, softplus, limit, groups, act)
    drow, dring, dstate = row.cuda(), ring.cuda(), state.cuda()
    out = binding.conv1d_ssd_update(drow[:, hp:hp + ch], drow[:, hp + ch:], A.cuda(), w.cuda(), dring, dstate, _ints(seen),
                                    conv_bias=b.cuda(), D=D.cuda(), z=drow[:, :hp] if kw.get("z") else None,
                                    dt_bias=bias.cuda(), dt_softplus=softplus, dt_limit=limit, slots=_ints(slots),
                                    activation=act)
    R.close(out, ref, mag, io, "out", STEP)
    R.close(dstate, state1, statem, f32, "state", STEP)
    assert torch.equal(dring.cpu(), ring1), "ring"


@pytest.mark.parametrize("batch", [1, 40, 300])
def test_step_batches(batch):
    """Every split of a head's channels, without optional inputs."""
    log(f"[step] batch={batch}")
    g, heads, n = _gen(batch), 4, 64
    ch = heads * R.P + 2 * n
    xbc, dt = _randn(g, batch, ch, dtype=bf), _randn(g, batch, heads, dtype=bf) - 3
    w, A = _randn(g, ch, 4, scale=0.5), -1 - 7 * torch.rand(heads, generator=g)
    seen = [i % 6 for i in range(batch)]
    ring, state = _randn(g, batch, ch, 4, dtype=bf), _randn(g, batch, heads, R.P, n)
    ref, mag, ring1, state1, statem = _step_ref(xbc, dt, A, w, ring, state, seen, list(range(batch)), torch.zeros(ch),
                                                torch.zeros(heads), None, None, True, None, 1, True)
    dring, dstate = ring.cuda(), state.cuda()
    out = binding.conv1d_ssd_update(xbc.cuda(), dt.cuda(), A.cuda(), w.cuda(), dring, dstate, _ints(seen), dt_softplus=True)
    R.close(out, ref, mag, bf, "out", STEP)
    R.close(dstate, state1, statem, f32, "state", STEP)
    assert torch.equal(dring.cpu(), ring1)


# ---- together -------------------------------------------------------------

def test_prompt_then_tokens():
    """A prompt in two parts and single tokens leave the caches that the whole
    sequence in one call leaves."""
    log("[together] prompt then tokens")
    g, heads, G, n, T = _gen(1), 4, 2, 64, 150
    hp, ch = heads * R.P, heads * R.P + 2 * G * n
    xbc, dt = _randn(g, T, ch, dtype=bf).cuda(), (_randn(g, T, heads, dtype=bf) - 3).cuda()
    w, b, A, D = (v.cuda() for v in (_randn(g, ch, 4, scale=0.5), _randn(g, ch), -1 - 7 * torch.rand(heads, generator=g), _randn(g, heads)))

    def prompt(lo, hi, ring, state):
        seen, cu = _ints([lo]), _ints([0, hi - lo])
        u = binding.causal_conv1d_varlen_fwd(xbc[lo:hi], w, cu, bias=b, activation="silu", conv_state=ring, cache_seqlens=seen)
        return binding.ssd_varlen_fwd(u[:, :hp].view(-1, heads, R.P), dt[lo:hi], A, u[:, hp:hp + G * n].view(-1, G, n),
                                      u[:, hp + G * n:].view(-1, G, n), cu, hi - lo, D=D, dt_softplus=True, ssm_state=state,
                                      cache_seqlens=seen)

    caches = [(torch.full((1, ch, 4), float("nan"), dtype=bf, device="cuda"),
               torch.full((1, heads, R.P, n), float("nan"), device="cuda")) for _ in range(2)]
    whole = prompt(0, T, *caches[0])
    parts = [prompt(0, 70, *caches[1]), prompt(70, 145, *caches[1])]
    for t in range(145, T):
        parts.append(binding.conv1d_ssd_update(xbc[t:t + 1], dt[t:t + 1], A, w, *caches[1], _ints([t]), conv_bias=b, D=D,
                                               dt_softplus=True).view(1, heads, R.P))
    assert torch.equal(caches[0][0], caches[1][0])
    # the prompt's conv output is rounded to bf16, the step's is not: 2^-8 for each of x, B and C, over the terms
    parts = torch.cat(parts).float()
    scale = whole.float().square().mean().sqrt()
    assert (parts[:145] - whole[:145].float()).abs().max() <= 2.0 ** -7 * whole.float().abs().max()
    assert (parts[145:] - whole[145:].float()).square().mean().sqrt() <= 4 * 2.0 ** -8 * scale
    a, c = caches[0][1], caches[1][1]
    assert (a - c).square().mean().sqrt() <= 2 * 2.0 ** -8 * a.square().mean().sqrt()


def test_another_stream():
    t, cu = _scan_case(3, (100, 30), 4, 1, 64)
    d, kw = _call(t)
    cu, args = _ints(cu), dict(D=d["D"], dt_bias=d["dt_bias"])
    want = binding.ssd_varlen_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], cu, 100, **args, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = binding.ssd_varlen_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], cu, 100, **args, **kw)
    side.synchronize()
    assert torch.equal(want, got)


def test_captured_training_step():
    """Forward, backward and the conv's backward in a graph, replayed between
    eager calls and synchronisations."""
    log("[together] graph")
    t, cu = _scan_case(6, (130, 62), 4, 1, 64)
    d, kw = _call(t)
    cu, T = _ints(cu), 192
    codes = torch.zeros(binding.ssd_checkpoint_slots(T, 2), 4, R.P, 64, dtype=torch.int8, device="cuda")
    scales = torch.ones(codes.shape[:3], device="cuda")
    dout, w = _randn(_gen(8), T, 4, R.P, dtype=bf).cuda(), _randn(_gen(9), 256, 4).cuda()

    def step():
        args = (d["x"], d["dt"], d["A"], d["B"], d["C"], cu, 130)
        out = binding.ssd_varlen_fwd(*args, D=d["D"], dt_bias=d["dt_bias"], checkpoints=(codes, scales), **kw)
        g = binding.ssd_varlen_bwd(*args, dout, (codes, scales), D=d["D"], dt_bias=d["dt_bias"], **kw)
        c = binding.causal_conv1d_varlen_bwd(d["x"].view(T, 256), w, cu, g["dx"].view(T, 256), activation="silu")
        return [out] + [g[k] for k in sorted(g)] + [c["dx"], c["dweight"]]

    want = [v.clone() for v in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        for v in got:
            v.zero_()
        codes.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        for a, b in zip(want, step()):
            assert torch.equal(a, b)


def test_example_trains_and_serves():
    log("[together] example")
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mamba2_mixer.py")
    spec = importlib.util.spec_from_file_location("mamba2_mixer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    mixer = ex.Mixer()
    losses = ex.train(mixer, steps=20)
    assert losses[-1] < 0.7 * losses[0], losses
    got, want = ex.serve(mixer)
    # bf16 activations: the step's conv output is not rounded, its gate is inside; a few roundings of 2^-8
    assert (got.float() - want.float()).norm() <= 8 * 2.0 ** -8 * want.float().norm()


# ---- far offsets and broadcast inputs -------------------------------------

def test_offsets_past_32_bits():
    """Cache entries and tokens whose byte offsets pass 2^32 (and element
    offsets 2^31): the last entry of a cache of 9 GB, rows 9 MB apart."""
    log("[far] cache entry")
    h, n, entries = 80, 128, 3400
    state = torch.empty(entries, h, R.P, n, device="cuda")
    assert state.numel() > 1 << 31
    g = _gen(2)
    t, cu = _scan_case(2, (70,), h, 1, n)
    first = _randn(g, 1, h, R.P, n)
    state[entries - 1] = first[0].cuda()
    ref, mag, last, lastm, _ = R.scan_fwd(t, cu, first)
    d, kw = _call(t)
    out = binding.ssd_varlen_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), 70, D=d["D"], dt_bias=d["dt_bias"],
                                 ssm_state=state, cache_seqlens=_ints([9]), slots=_ints([entries - 1]), **kw)
    R.close(out, ref, mag, bf, "out")
    R.close(state[entries - 1:], last, lastm, f32, "state")
    ch = h * R.P + 2 * n
    xbc, dt = _randn(g, 1, ch, dtype=bf), _randn(g, 1, h, dtype=bf) - 3
    w, A = _randn(g, ch, 4, scale=0.5), -1 - torch.rand(h, generator=g)
    ring = torch.zeros(entries, ch, 4, dtype=bf, device="cuda")
    ref, mag, _, state1, statem = _step_ref(xbc, dt, A, w, ring[-1:].cpu(), state[-1:].cpu(), [3], [0], torch.zeros(ch),
                                            torch.zeros(h), None, None, True, None, 1, True)
    out = binding.conv1d_ssd_update(xbc.cuda(), dt.cuda(), A.cuda(), w.cuda(), ring, state, _ints([3]), dt_softplus=True,
                                    slots=_ints([entries - 1]))
    R.close(out, ref, mag, bf, "step out", STEP)
    R.close(state[entries - 1:], state1, statem, f32, "step state", STEP)
    del state, ring
    log("[far] tokens")
    row, T = 1 << 22, 600
    far = torch.zeros(T, row, dtype=bf, device="cuda")
    assert far.numel() > 1 << 31
    t, cu = _scan_case(4, (T,), 2, 1, 32)
    d, kw = _call(t)
    x = far[:, 8:8 + 128].view(T, 2, R.P)
    x.copy_(d["x"])
    ref, mag, *_ = R.scan_fwd(t, cu)
    out = binding.ssd_varlen_fwd(x, d["dt"], d["A"], d["B"], d["C"], _ints(cu), T, D=d["D"], dt_bias=d["dt_bias"], **kw)
    R.close(out, ref, mag, bf, "far x")
    w = _randn(g, 128, 4)
    ref, mag, _ = R.conv_fwd(t["x"].view(T, 128), w, None, cu, True)
    got = binding.causal_conv1d_varlen_fwd(far[:, 8:8 + 128], w.cuda(), _ints(cu), activation="silu", out=far[:, 1024:1024 + 128])
    R.close(got, ref, mag, bf, "far conv", R.SHORT)


def test_broadcast_inputs():
    """Inputs expanded over tokens, groups or heads: gradients of the expanded
    tensors, as for dense ones."""
    t, cu = _scan_case(4, (70, 3), 4, 2, 32)
    t["B"], t["A"] = t["B"][:, :1].expand(-1, 2, -1), t["A"][:1].expand(4)
    d, kw = _call(t)
    codes = torch.zeros(binding.ssd_checkpoint_slots(73, 2), 4, R.P, 32, dtype=torch.int8, device="cuda")
    scales = torch.ones(codes.shape[:3], device="cuda")
    dout = _randn(_gen(1), 1, 4, R.P, dtype=bf).expand(73, -1, -1)
    B, A = t["B"][:, :1].contiguous().cuda().expand(-1, 2, -1), t["A"][:1].contiguous().cuda().expand(4)
    args = (d["x"], d["dt"], A, B, d["C"], _ints(cu), 70)
    binding.ssd_varlen_fwd(*args, D=d["D"], dt_bias=d["dt_bias"], checkpoints=(codes, scales), **kw)
    got = binding.ssd_varlen_bwd(*args, dout[:1].contiguous().cuda().expand(73, -1, -1), (codes, scales), D=d["D"],
                                 dt_bias=d["dt_bias"], **kw)
    ref = R.scan_bwd(t, cu, dout, codes.cpu(), scales.cpu())
    for k in ("dx", "ddt", "dB", "dC"):
        R.close(got[k], *ref[k], bf, k)
    for k in ("dA", "dD", "ddt_bias"):
        R.close(got[k], *ref[k], f32, k)


def test_refused_on_the_gpu():
    """What needs device tensors to be refused: outputs that are not writable in
    place, and a workspace that is too small."""
    t, cu = _scan_case(4, (200,), 2, 1, 32)
    d, kw = _call(t)
    args = (d["x"], d["dt"], d["A"], d["B"], d["C"], _ints(cu), 200)
    with pytest.raises(ValueError, match="written in place"):
        binding.ssd_varlen_fwd(*args, out=torch.empty(2, 200, R.P, dtype=bf, device="cuda").transpose(0, 1), **kw)
    with pytest.raises(ValueError, match="status 5"):
        binding.ssd_varlen_fwd(*args, seq_segments=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **kw)
    with pytest.raises(ValueError, match="status 3"):
        bad = torch.zeros(200, 1, 48, dtype=bf, device="cuda")
        binding.ssd_varlen_fwd(d["x"], d["dt"], d["A"], bad, bad, _ints(cu), 200, **kw)
