"""The gated linear recurrence, its gradient, its step and the norm on the GPU
against the 64-bit references of gated_ref.py (whose head derives the bounds)."""
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


def _case(seed, T, C, io, bias=True, slow=False):
    g = torch.Generator().manual_seed(seed)
    t = dict(x=_randn(g, T, C, dtype=io), r=_randn(g, T, C, dtype=io), i=_randn(g, T, C, dtype=io),
             A=-(0.001 if slow else 1.0) * (0.05 + 3 * torch.rand(C, generator=g)),
             r_bias=_randn(g, C, scale=0.5) if bias else None, i_bias=_randn(g, C, scale=0.5) if bias else None)
    return t, g


def _dev(t):
    return [t[k].cuda() for k in ("x", "r", "i", "A")], {k: t[k].cuda() for k in ("r_bias", "i_bias") if t[k] is not None}


LENS = [(1,), (64,), (65,), (5, 0, 1, 130), (0, 0, 3, 63, 1, 64, 2, 0), (300, 1, 0, 211), (1,) * 70, (700,)]


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("C", [8, 67, 264])
@pytest.mark.parametrize("lens", LENS)
def test_scan_fwd(io, C, lens):
    log(f"[gated fwd] {io} C={C} lens={lens}")
    cu = R.sequences(lens)
    t, _ = _case(C + sum(lens), cu[-1], C, io)
    args, kw = _dev(t)
    ref = R.scan(t, cu)
    kept = torch.full((-(-cu[-1] // 64), C), float("nan"), device="cuda")
    out = binding.gated_scan_varlen_fwd(*args, _ints(cu), checkpoints=kept, **kw)
    R.close(out, ref["after"], ref["err"], io, "out")
    R.close(kept, ref["before"][::64], ref["err_before"][::64], f32, "kept states")
    assert torch.equal(out, binding.gated_scan_varlen_fwd(*args, _ints(cu), **kw)), "without kept states"
    t.update(r_bias=None, i_bias=None)
    ref = R.scan(t, cu)
    R.close(binding.gated_scan_varlen_fwd(*args, _ints(cu)), ref["after"], ref["err"], io, "out without biases")


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("C", [40, 129])
def test_scan_fwd_cache(io, C):
    """From and to a cache, with inputs and outputs that are parts of wider rows."""
    lens, seen, slots = (5, 1, 0, 200, 30, 3, 9, 70), [0, 1, 2, 3, 0, 1000, 2, 7], [6, 2, 0, 7, 1, -1, 99, 3]
    log(f"[gated cache] {io} C={C}")
    cu = R.sequences(lens)
    t, g = _case(C, cu[-1], C, io)
    (x, r, i, A), kw = _dev(t)
    cache = _randn(g, 8, C)
    cache[6] = float("nan")   # a new request's entry is never looked at
    ref, err, after, e_after = R.scan_cached(t, cu, cache, seen, slots)
    wide = torch.full((cu[-1], 3 * C + 8), float("nan"), dtype=io, device="cuda")
    parts = [wide[:, k * C:(k + 1) * C] for k in range(3)]
    for p, v in zip(parts, (x, r, i)):
        p.copy_(v)
    room = torch.zeros(cu[-1], C + 6, dtype=io, device="cuda")
    state = cache.cuda()
    out = binding.gated_scan_varlen_fwd(*parts, A, _ints(cu), state=state, cache_seqlens=_ints(seen), slots=_ints(slots),
                                        out=room[:, 6:], **kw)
    R.close(out, ref, err, io, "out")
    R.close(state, after, e_after, f32, "cache")
    assert not room[:, :6].any()
    assert torch.equal(state[[0, 4, 5]].cpu(), cache[[0, 4, 5]]), "entries of no token"
    # no cache_seqlens: every request is new; no slots: sequence s is entry s
    state = torch.full((8, C), float("nan"), device="cuda")
    out = binding.gated_scan_varlen_fwd(x, r, i, A, _ints(cu), state=state, **kw)
    ref = R.scan(t, cu)
    R.close(out, ref["after"], ref["err"], io, "out of new requests")
    assert torch.isnan(state[2]).all()
    keep = [0, 1, 3, 4, 5, 6, 7]
    R.close(state[keep], ref["last"][keep], ref["last_err"][keep], f32, "cache of new requests")


def test_scan_fwd_of_many_tokens():
    """A memory of thousands of tokens: slow decay over tiles and groups of them."""
    lens = (3000, 5, 4200)
    cu = R.sequences(lens)
    t, g = _case(1, cu[-1], 96, f32, slow=True)
    args, kw = _dev(t)
    state = _randn(g, 3, 96)
    ref, err, after, e_after = R.scan_cached(t, cu, state, [1, 1, 1], [0, 1, 2])
    dstate = state.cuda()
    out = binding.gated_scan_varlen_fwd(*args, _ints(cu), state=dstate, cache_seqlens=_ints([1, 1, 1]), **kw)
    log(f"[gated long] largest relative error {((out.cpu().double() - ref).norm() / ref.norm()):.2e}")
    R.close(out, ref, err, f32, "out")
    R.close(dstate, after, e_after, f32, "cache")


def test_scan_continues_what_it_left():
    """A prompt in two calls and then single tokens is the whole sequence."""
    C, lens = 130, (70, 3, 129)
    t, _ = _case(4, sum(lens), C, f32)
    cu = R.sequences(lens)
    (x, r, i, A), kw = _dev(t)
    ref = R.scan(t, cu)
    state, slots = torch.full((5, C), float("nan"), device="cuda"), _ints([4, 0, 2])
    cut, got = [40, 1, 128], [[] for _ in lens]

    def part(lo, hi):
        rows = torch.cat([torch.arange(cu[s] + lo[s], cu[s] + hi[s]) for s in range(3)]).cuda()
        n = [hi[s] - lo[s] for s in range(3)]
        out = binding.gated_scan_varlen_fwd(x[rows], r[rows], i[rows], A, _ints(R.sequences(n)), state=state,
                                            cache_seqlens=_ints(lo), slots=slots, **kw)
        for s, v in enumerate(out.split(n)):
            got[s].append(v)

    part([0, 0, 0], cut)
    part(cut, [min(n, c + 20) for n, c in zip(lens, cut)])
    at = [min(n, c + 20) for n, c in zip(lens, cut)]
    while any(a < n for a, n in zip(at, lens)):   # single tokens, padding for who is done
        alive = [a < n for a, n in zip(at, lens)]
        rows = torch.tensor([cu[s] + min(at[s], lens[s] - 1) for s in range(3)]).cuda()
        out = binding.gated_scan_update(x[rows], r[rows], i[rows], A, state, _ints(at),
                                        slots=torch.where(torch.tensor(alive).cuda(), slots, -1).to(i32), **kw)
        for s in range(3):
            if alive[s]:
                got[s].append(out[s:s + 1])
                at[s] += 1
    R.close(torch.cat([torch.cat(v) for v in got]), ref["after"], ref["err"], f32, "out")


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("C", [8, 67, 264])
@pytest.mark.parametrize("lens", LENS)
def test_scan_bwd(io, C, lens):
    log(f"[gated bwd] {io} C={C} lens={lens}")
    cu = R.sequences(lens)
    t, g = _case(C + sum(lens), cu[-1], C, io)
    dout = _randn(g, cu[-1], C, dtype=io)
    args, kw = _dev(t)
    kept = torch.empty(-(-cu[-1] // 64), C, device="cuda")
    binding.gated_scan_varlen_fwd(*args, _ints(cu), checkpoints=kept, **kw)
    got = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, **kw)
    ref = R.scan_bwd(t, cu, dout)
    assert set(got) == {"dx", "dr", "di", "dA", "dr_bias", "di_bias"}
    for k, v in got.items():
        R.close(v, *ref[k], io if k in ("dx", "dr", "di") else f32, k)
    again = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, **kw)
    for k, v in got.items():
        assert torch.equal(v, again[k]), f"{k} repeats"


@pytest.mark.parametrize("io", [f32, bf])
def test_scan_bwd_states_and_strides(io):
    """Initial and final states' gradients, no biases, gradients as parts of a row."""
    lens, C = (130, 0, 1, 64, 7, 0), 72
    cu = R.sequences(lens)
    t, g = _case(11, cu[-1], C, io, bias=False)
    (x, r, i, A), _ = _dev(t)
    h0, dfin, dout = _randn(g, 6, C), _randn(g, 6, C), _randn(g, cu[-1], C, dtype=io)
    kept = torch.empty(-(-cu[-1] // 64), C, device="cuda")
    state = h0.cuda()
    binding.gated_scan_varlen_fwd(x, r, i, A, _ints(cu), state=state, cache_seqlens=_ints([1] * 6), checkpoints=kept)
    row = torch.zeros(cu[-1], 3 * C + 4, dtype=io, device="cuda")
    dx, dr, di = (row[:, 4 + k * C:4 + (k + 1) * C] for k in range(3))
    got = binding.gated_scan_varlen_bwd(x, r, i, A, _ints(cu), dout.cuda(), kept, initial_states=h0.cuda(),
                                        dfinal_states=dfin.cuda(), want_dinitial_states=True, dx=dx, dr=dr, di=di)
    ref = R.scan_bwd(t, cu, dout, h0, dfin)
    assert set(got) == {"dx", "dr", "di", "dA", "dinitial_states"}
    for k, v in got.items():
        R.close(v, *ref[k], io if k in ("dx", "dr", "di") else f32, k)
    assert got["dx"].data_ptr() == dx.data_ptr() and not row[:, :4].any()


def test_scan_bwd_of_many_tokens():
    lens = (2500, 3, 1900)
    cu = R.sequences(lens)
    t, g = _case(2, cu[-1], 96, f32, slow=True)
    dout = _randn(g, cu[-1], 96)
    args, kw = _dev(t)
    kept = torch.empty(-(-cu[-1] // 64), 96, device="cuda")
    binding.gated_scan_varlen_fwd(*args, _ints(cu), checkpoints=kept, **kw)
    got = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, **kw)
    ref = R.scan_bwd(t, cu, dout)
    for k, v in got.items():
        log(f"[gated bwd long] {k} {((v.cpu().double() - ref[k][0]).norm() / ref[k][0].norm()):.2e}")
        R.close(v, *ref[k], f32, k)


# (as a call is cut: by tokens and channels; sequences that end anywhere, and more of them than a wave has lanes)
CUTS = [(4200, 1030, 5), (3100, 4097, 3), (1700, 200, 3), (900, 1000, 200), (130, 1000, 2)]


@pytest.mark.parametrize("io", [f32, bf])
@pytest.mark.parametrize("T,C,nseq", CUTS)
def test_every_cut(io, T, C, nseq):
    log(f"[gated cuts] {io} {T}x{C} in {nseq}")
    t, g = _case(T + C, T, C, io)
    cuts = sorted(torch.randint(0, T + 1, (nseq - 1,), generator=g).tolist())
    cu = [0] + cuts + [T]
    dout = _randn(g, T, C, dtype=io)
    state, slots = _randn(g, nseq, C), torch.randperm(nseq, generator=g).tolist()
    args, kw = _dev(t)
    kept, dstate = torch.empty(-(-T // 64), C, device="cuda"), state.cuda()
    out = binding.gated_scan_varlen_fwd(*args, _ints(cu), state=dstate, cache_seqlens=_ints([1] * nseq), slots=_ints(slots),
                                        checkpoints=kept, **kw)
    ref, err, after, e_after = R.scan_cached(t, cu, state, [1] * nseq, slots)
    R.close(out, ref, err, io, "out")
    R.close(dstate, after, e_after, f32, "cache")
    h0 = state[slots]
    dfin = _randn(g, nseq, C)
    got = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, initial_states=h0.cuda(), dfinal_states=dfin.cuda(),
                                        want_dinitial_states=True, **kw)
    want = R.scan_bwd(t, cu, dout, h0, dfin)
    for k, v in got.items():
        R.close(v, *want[k], io if k in ("dx", "dr", "di") else f32, k)


@pytest.mark.parametrize("C", [72, 65])
def test_padding(C):
    """Tokens before the first sequence and behind the last: their outputs stay,
    their gradients are 0, and what they hold reaches nothing."""
    lens, first, tail = (70, 0, 5, 130), 67, 140
    cu = R.sequences(lens, first)
    T = cu[-1] + tail
    t, g = _case(5, T, C, bf)
    for k in ("x", "r", "i"):
        t[k][:first] = float("nan")
        t[k][cu[-1]:] = float("inf")
    dout = _randn(g, T, C, dtype=bf)
    dout[:first], dout[cu[-1]:] = float("inf"), float("nan")
    args, kw = _dev(t)
    kept = torch.full((-(-T // 64), C), float("nan"), device="cuda")
    out = torch.full((T, C), 7.0, dtype=bf, device="cuda")
    state = torch.zeros(4, C, device="cuda")
    binding.gated_scan_varlen_fwd(*args, _ints(cu), state=state, checkpoints=kept, out=out, **kw)
    clean = {k: v if v is None or v.dim() == 1 else torch.nan_to_num(v, 0.0, 0.0, 0.0) for k, v in t.items()}
    ref = R.scan(clean, cu)
    inside = slice(first, cu[-1])
    R.close(out[inside], ref["after"][inside], ref["err"][inside], bf, "out")
    assert (out[:first] == 7).all() and (out[cu[-1]:] == 7).all()
    R.close(kept, ref["before"][::64], ref["err_before"][::64], f32, "kept states")
    R.close(state, ref["last"], ref["last_err"], f32, "cache")
    got = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, want_dinitial_states=True, **kw)
    want = R.scan_bwd(clean, cu, torch.nan_to_num(dout, 0.0, 0.0, 0.0))
    for k, v in got.items():
        R.close(v, *want[k], bf if k in ("dx", "dr", "di") else f32, k)
    for k in ("dx", "dr", "di"):
        assert not got[k][:first].any() and not got[k][cu[-1]:].any()


def test_nothing_but_padding():
    x = torch.ones(70, 16, dtype=bf, device="cuda")
    A, cu = -torch.ones(16, device="cuda"), _ints([70, 70, 70])
    out, kept, state = torch.full_like(x, 3.0), torch.ones(2, 16, device="cuda"), torch.full((2, 16), 5.0, device="cuda")
    binding.gated_scan_varlen_fwd(x, x, x, A, cu, out=out, checkpoints=kept, state=state)
    assert (out == 3).all() and not kept.any() and (state == 5).all()
    dfin = torch.randn(2, 16, device="cuda")
    got = binding.gated_scan_varlen_bwd(x, x, x, A, cu, x, kept, dfinal_states=dfin, want_dinitial_states=True)
    assert torch.equal(got.pop("dinitial_states"), dfin)
    for k, v in got.items():
        assert not v.any(), k


def test_scan_keeps_to_its_sequence():
    """Infinities and NaN stay in their sequence and channel, and in the forward
    behind their token; a later sequence starts clean."""
    cu = [0, 100, 190, 400]
    t, g = _case(6, 400, 40, f32)
    dout = _randn(g, 400, 40)
    for k, v in (("x", float("inf")), ("r", float("nan")), ("i", float("-inf"))):
        t[k][130, :7] = v
    args, kw = _dev(t)
    kept = torch.empty(7, 40, device="cuda")
    out = binding.gated_scan_varlen_fwd(*args, _ints(cu), checkpoints=kept, **kw)
    got = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, **kw)
    bad = torch.zeros(400, 40, dtype=torch.bool)
    bad[130:190, :7] = True
    assert torch.isfinite(out.cpu()[~bad]).all() and torch.isnan(out.cpu()[bad]).all()
    for k in ("dx", "dr", "di"):
        v = got[k].cpu()
        assert torch.isfinite(v[:100]).all() and torch.isfinite(v[190:]).all() and torch.isfinite(v[:, 7:]).all()
    for k in ("dA", "dr_bias", "di_bias"):
        assert torch.isfinite(got[k].cpu()[7:]).all()


def test_gates_at_their_ends():
    """Gates far open and far closed, a state that is only kept, and A of 0 or above."""
    T, C = 130, 8
    x, r, i = torch.randn(T, C, device="cuda"), torch.zeros(T, C, device="cuda"), torch.zeros(T, C, device="cuda")
    A = torch.tensor([-1.0, -1.0, 0.0, 0.01, -200.0, -1.0, -1e-30, -1.0], device="cuda")
    r[:, 0], r[:, 1], i[:, 5], i[:, 7] = 200.0, -200.0, -200.0, 200.0
    state = torch.ones(1, C, device="cuda")
    kept = torch.empty(3, C, device="cuda")
    out = binding.gated_scan_varlen_fwd(x, r, i, A, _ints([0, T]), state=state, cache_seqlens=_ints([1]), checkpoints=kept)
    assert torch.isfinite(out).all()
    assert (out[:, 1] == 1).all() and (out[:, 2] == 1).all(), "a closed gate keeps the state"
    assert torch.allclose(out[:, 3].cpu(), torch.exp(0.005 * torch.arange(1, T + 1)), rtol=1e-5)
    assert torch.allclose(out[:, 4], torch.sigmoid(i[:, 4]) * x[:, 4], rtol=1e-6)
    assert torch.allclose(out[:, 5].cpu(), torch.exp(-0.5 * torch.arange(1, T + 1)), rtol=1e-4, atol=1e-30)
    got = binding.gated_scan_varlen_bwd(x, r, i, A, _ints([0, T]), x, kept, initial_states=torch.ones(1, C, device="cuda"))
    for k, v in got.items():
        assert torch.isfinite(v).all(), k


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("B,C", [(1, 8), (3, 67), (33, 2560), (70, 520)])
def test_update(io, B, C):
    log(f"[gated update] {io} B={B} C={C}")
    t, g = _case(B + C, B, C, io)
    (x, r, i, A), kw = _dev(t)
    cache = _randn(g, B + 3, C)
    slots = torch.randperm(B + 3, generator=g)[:B].tolist()
    seen = [k % 3 for k in range(B)]
    if B > 2:
        slots[1], slots[2] = -1, B + 3
    for s, n in zip(slots, seen):
        if n == 0 and 0 <= s < B + 3:
            cache[s] = float("nan")
    ref, err, after, e_after = R.scan_cached(t, list(range(B + 1)), cache, seen, slots)
    state = cache.cuda()
    room = torch.zeros(B, C + 3, dtype=io, device="cuda")
    out = binding.gated_scan_update(x, r, i, A, state, _ints(seen), slots=_ints(slots), out=room[:, 3:], **kw)
    R.close(out, ref, err, io, "out")
    used = sorted(s for s in slots if 0 <= s < B + 3)
    rest = [s for s in range(B + 3) if s not in used]
    R.close(state[used], after[used], e_after[used], f32, "cache")
    assert torch.equal(state[rest].cpu(), cache[rest]) and not room[:, :3].any()
    # every request new, entry b for request b
    ref = R.scan(t, list(range(B + 1)))
    out = binding.gated_scan_update(x, r, i, A, state, None, **kw)
    R.close(out, ref["after"], ref["err"], io, "out of new requests")
    R.close(state[:B], ref["last"], ref["last_err"], f32, "cache of new requests")


# ---- norm -------------------------------------------------------------------

SHAPES = [(1, 8, 8), (5, 1, 1), (3, 67, 67), (70, 128, 128), (9, 520, 104), (33, 2560, 2560), (4, 1001, 143), (2, 5120, 640),
          (300, 40, 8), (2, 16384, 16384), (3, 9001, 9001), (6, 4096, 512)]


def _norm_case(seed, T, C, io, kind):
    g = torch.Generator().manual_seed(seed)
    res = {"same": io, "wide": f32}.get(kind)
    x, w = _randn(g, T, C, dtype=io), 1 + 0.3 * _randn(g, C)
    return g, x, w, None if res is None else _randn(g, T, C, dtype=res, scale=3.0), _randn(g, T, C, dtype=io) if kind == "gate" else None


def _cuda(v):
    return None if v is None else v.cuda()


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("kind", ["plain", "same", "wide", "gate"])
@pytest.mark.parametrize("T,C,n", SHAPES)
def test_norm_fwd(io, kind, T, C, n):
    log(f"[norm fwd] {io} {kind} {T}x{C} groups of {n}")
    _, x, w, res, z = _norm_case(T + C, T, C, io, kind)
    ref, err, held = R.norm(x, w, res, z, n)
    got = binding.rms_norm_fwd(x.cuda(), w.cuda(), residual=_cuda(res), z=_cuda(z), group_size=n)
    out, kept = got if res is not None else (got, None)
    R.close(out, ref, err, io, "out")
    if res is not None:
        assert torch.equal(kept.cpu(), held), "residual"
        stream = res.cuda()   # in place
        out2, same = binding.rms_norm_fwd(x.cuda(), w.cuda(), residual=stream, group_size=n, residual_out=stream)
        assert same.data_ptr() == stream.data_ptr() and torch.equal(stream, kept) and torch.equal(out2, out)


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("kind", ["plain", "same", "wide", "gate"])
@pytest.mark.parametrize("T,C,n", [(1, 8, 8), (3, 67, 67), (70, 128, 128), (33, 2560, 2560), (5, 2560, 640), (4, 1001, 1001),
                                   (2, 16384, 16384), (3, 9001, 9001), (6, 4096, 512), (300, 136, 136)])
def test_norm_quant(io, kind, T, C, n):
    log(f"[norm quant] {io} {kind} {T}x{C} groups of {n}")
    _, x, w, res, z = _norm_case(T + C + 1, T, C, io, kind)
    x[0, :min(C, 40)] *= 100   # a block of another size than its neighbours
    if T > 2:
        x[2] = 0
        if res is not None:
            res[2] = 0
    ref, err, held = R.norm(x, w, res, z, n)
    codes, scales, *kept = binding.rms_norm_quant_fwd(x.cuda(), w.cuda(), residual=_cuda(res), z=_cuda(z), group_size=n)
    assert codes.dtype == torch.float8_e4m3fn and scales.shape == (T, -(-C // 128))
    if res is not None:
        assert torch.equal(kept[0].cpu(), held)
    s = scales.cpu().double()
    frac, _ = torch.frexp(s)
    assert (frac == 0.5).all() and (s >= 2.0 ** -100).all()
    wide = s.repeat_interleave(128, 1)[:, :C]
    value = codes.cpu().float().double() * wide
    assert torch.isfinite(value).all()
    tol = R.e4m3_step(ref.abs() + err, wide) + err
    assert ((value - ref).abs() <= tol).all(), f"over by {((value - ref).abs() - tol).max():.3e}"
    pad = torch.nn.functional.pad(ref.abs(), (0, -C % 128)).view(T, -1, 128).amax(-1)
    slack = torch.nn.functional.pad(err, (0, -C % 128)).view(T, -1, 128).amax(-1)
    assert (pad - slack <= 448 * s).all(), "a scale too small"
    assert ((pad + slack > 224 * s) | (s == 2.0 ** -100)).all(), "a scale too large"


@pytest.mark.parametrize("io", [f32, bf, f16])
@pytest.mark.parametrize("kind", ["plain", "same", "wide", "gate"])
@pytest.mark.parametrize("T,C,n", SHAPES)
def test_norm_bwd(io, kind, T, C, n):
    log(f"[norm bwd] {io} {kind} {T}x{C} groups of {n}")
    g, x, w, res, z = _norm_case(T + C + 2, T, C, io, kind)
    s = x if res is None else (x.float() + res.float()).to(res.dtype)
    dy = _randn(g, T, C, dtype=io)
    ds = None if res is None else _randn(g, T, C, dtype=res.dtype)
    ref = R.norm_bwd(s, w, dy, z, ds, n)
    got = binding.rms_norm_bwd(s.cuda(), w.cuda(), dy.cuda(), z=_cuda(z), ds=_cuda(ds), group_size=n)
    want = {"dx", "dweight"} | ({"dz"} if z is not None else set()) | ({"dresidual"} if s.dtype != io else set())
    assert set(got) == want
    for k, v in got.items():
        R.close(v, *ref[k], {"dweight": f32, "dresidual": f32}.get(k, io), k)
    if res is not None:   # the gradient without the stream's
        alone = binding.rms_norm_bwd(s.cuda(), w.cuda(), dy.cuda(), group_size=n)
        R.close(alone["dx"], *R.norm_bwd(s, w, dy, None, None, n)["dx"], io, "dx alone")


@pytest.mark.parametrize("io,kind,T,C,n", [(bf, "wide", 3000, 512, 512), (bf, "gate", 2100, 640, 80), (f32, "same", 1500, 129, 43)])
def test_norm_bwd_of_many_rows(io, kind, T, C, n):
    log(f"[norm bwd many] {io} {kind} {T}x{C}")
    g, x, w, res, z = _norm_case(7, T, C, io, kind)
    s = x if res is None else (x.float() + res.float()).to(res.dtype)
    dy, ds = _randn(g, T, C, dtype=io), None if res is None else _randn(g, T, C, dtype=res.dtype)
    ref = R.norm_bwd(s, w, dy, z, ds, n)
    args, kw = (s.cuda(), w.cuda(), dy.cuda()), dict(z=_cuda(z), ds=_cuda(ds), group_size=n)
    got, again = binding.rms_norm_bwd(*args, **kw), binding.rms_norm_bwd(*args, **kw)
    for k, v in got.items():
        R.close(v, *ref[k], {"dweight": f32, "dresidual": f32}.get(k, io), k)
        assert torch.equal(v, again[k])


@pytest.mark.parametrize("kind", ["same", "gate"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_norm_strides(kind, shift):
    """Inputs and outputs that are parts of wider rows, at any alignment."""
    T, C, n = 20, 1024, 512
    g, x, w, res, z = _norm_case(3, T, C, bf, kind)
    dy = _randn(g, T, C, dtype=bf)

    def part(v, fill=float("nan")):
        if v is None:
            return None
        wide = torch.full((T, C + 40), fill, dtype=v.dtype, device="cuda")
        wide[:, shift:shift + C] = v.cuda()
        return wide[:, shift:shift + C]

    ref, err, held = R.norm(x, w, res, z, n)
    room = torch.zeros(T, C + 9, dtype=bf, device="cuda")
    got = binding.rms_norm_fwd(part(x), w.cuda(), residual=part(res), z=part(z), group_size=n, out=room[:, shift:shift + C],
                               residual_out=part(res))
    R.close(got[0] if res is not None else got, ref, err, bf, "out")
    assert not room[:, :shift].any() and not room[:, shift + C:].any()
    if res is not None:
        assert torch.equal(got[1].cpu(), held)
    room8 = torch.zeros(T, C + 9, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    codes, scales, *_ = binding.rms_norm_quant_fwd(part(x), w.cuda(), residual=part(res), z=part(z), group_size=n,
                                                   codes=room8[:, shift:shift + C])
    dense = binding.rms_norm_quant_fwd(x.cuda(), w.cuda(), residual=_cuda(res), z=_cuda(z), group_size=n)
    assert torch.equal(scales, dense[1]) and torch.equal(codes.contiguous().view(torch.uint8), dense[0].view(torch.uint8))
    assert not room8.view(torch.uint8)[:, :shift].any()
    s = x if res is None else held
    ds = res
    want = R.norm_bwd(s, w, dy, z, ds, n)
    grads = binding.rms_norm_bwd(part(s), w.cuda(), part(dy), z=part(z), ds=part(ds), group_size=n, dx=part(dy, 0.0),
                                 dz=part(z, 0.0))
    for k, v in grads.items():
        R.close(v, *want[k], f32 if k == "dweight" else bf, k)


def test_norm_of_zeros_and_of_what_is_not_finite():
    x = torch.zeros(4, 300, dtype=bf, device="cuda")
    x[1, 3], x[2, 200] = float("inf"), float("nan")
    x[3] = 1
    w = torch.ones(300, device="cuda")
    out = binding.rms_norm_fwd(x, w)
    assert not out[0].any() and torch.isnan(out[2]).all() and torch.isfinite(out[3]).all()
    codes, scales = binding.rms_norm_quant_fwd(x, w)
    assert torch.isfinite(scales[0]).all() and torch.isfinite(scales[3]).all() and not codes[0].float().any()
    assert torch.isnan(scales[2]).all() and torch.isnan(scales[1, 0])
    got = binding.rms_norm_bwd(x, w, torch.ones_like(x))
    assert torch.isfinite(got["dx"][[0, 3]].float()).all()
