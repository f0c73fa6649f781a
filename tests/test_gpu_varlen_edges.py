"""Places where the packed-token operators can go wrong without their ordinary
tests seeing it: gradients that vanish, sequences that start at the end of a
run, edges outside the tokens, explicit streams.  References and tolerances as
in varlen_ref.py."""
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


def _ints(v):
    return torch.tensor(v, dtype=i32, device="cuda")


# ---- the decays' gradient -------------------------------------------------

def _steps_case(seed, lens, h, G, n, decay):
    """Positive steps, decays of about exp(-decay) a token, and the checkpoints
    of sequences that start from nothing."""
    g, T = _gen(seed), sum(lens)
    t = dict(x=_randn(g, T, h, R.P, dtype=bf), A=-decay * (0.5 + torch.rand(h, generator=g)), B=_randn(g, T, G, n, dtype=bf),
             C=_randn(g, T, G, n, dtype=bf), dt=(0.75 + 0.5 * torch.rand(T, h, generator=g)).to(bf))
    cu = R.sequences(lens)
    entries = binding.ssd_checkpoint_slots(T, len(lens))
    codes, scales = torch.full((entries, h, R.P, n), 3, dtype=torch.int8), torch.full((entries, h, R.P), float("nan"))
    for e, (S, _) in R.scan_fwd(t, cu)[4].items():
        codes[e], scales[e] = R.to_8_bits(S.float())
    return t, cu, _randn(g, T, h, R.P, dtype=bf), codes, scales, _randn(g, len(lens), h, R.P, n)


def _bwd(t, cu, dout, codes, scales, dlast):
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    return binding.ssd_varlen_bwd(*(t[k].cuda() for k in ("x", "dt", "A", "B", "C")), _ints(cu), longest, dout.cuda(),
                                  (codes.cuda(), scales.cuda()), dfinal_states=None if dlast is None else dlast.cuda())


def _through(t, cu, dout, codes, scales, dlast):
    """The gradient of every token's decay exponent, sum over its paths, and
    the sum of the paths' magnitudes: nothing in it cancels by construction."""
    x, B, C, A, g, d = (v.to(R.f64) for v in (t["x"], t["B"], t["C"], t["A"], dout, t["dt"]))
    rep = x.shape[1] // B.shape[1]
    up = lambda v: v.repeat_interleave(rep, 0)[:, None, :]  # noqa: E731
    keep = torch.exp(d * A)[..., None, None]
    da, dam = torch.zeros_like(d), torch.zeros_like(d)
    for s in range(len(cu) - 1):
        adj = torch.zeros(codes.shape[1:], dtype=R.f64) if dlast is None else dlast[s].to(R.f64).clone()
        adjm = adj.abs()
        for c in range((cu[s + 1] - cu[s] - 1) // R.Q, -1, -1):
            ks = range(cu[s] + c * R.Q, min(cu[s + 1], cu[s] + (c + 1) * R.Q))
            e = R.entry(cu, s, c)
            S = codes[e].to(R.f64) * scales[e].to(R.f64)[..., None]
            M, past = S.abs(), []
            for k in ks:
                past.append((S, M))
                add = (d[k][:, None] * x[k])[:, :, None] * up(B[k])
                S, M = keep[k] * S + add, keep[k] * M + add.abs()
            for k in reversed(ks):
                add = g[k][:, :, None] * up(C[k])
                adj, adjm = keep[k] * (adj + add), keep[k] * (adjm + add.abs())
                S, M = past[k - ks[0]]
                da[k], dam[k] = (adj * S).sum((1, 2)), (adjm * M).sum((1, 2))
    return da, dam


@pytest.mark.parametrize("n", [32, 64, 128])
@pytest.mark.parametrize("final", [False, True])
def test_no_decay_gradient_of_single_tokens(n, final):
    """A sequence of one token from nothing has no state that decays: dA is 0."""
    log(f"[decay] single tokens n={n} final={final}")
    *a, dlast = _steps_case(n, (1, 1, 0, 1, 1, 1), 6, 2, n, 1.0)
    got = _bwd(*a, dlast if final else None)
    assert torch.equal(got["dA"].cpu(), torch.zeros(6)), got["dA"]


@pytest.mark.parametrize("decay", [0.1, 1.0, 10.0])
@pytest.mark.parametrize("lens", [(2, 2, 1, 2), (17, 40), (64, 65), (200,)])
def test_decay_gradient_of_short_memories(lens, decay):
    """dA and ddt against the sum of their paths' magnitudes.  At exp(-10) a
    token a path through a decay weighs less than a rounding (2^-24) of the paths
    that do not pass one would, times the bound: those may not enter dA."""
    log(f"[decay] lens={lens} decay={decay}")
    t, cu, dout, codes, scales, dlast = _steps_case(3 + len(lens), lens, 4, 2, 64, decay)
    da, dam = _through(t, cu, dout, codes, scales, dlast)
    d = t["dt"].to(R.f64)
    got = _bwd(t, cu, dout, codes, scales, dlast)
    R.close(got["dA"], (d * da).sum(0), (d * dam).sum(0), f32, "dA")
    ref = R.scan_bwd(t, cu, dout, codes, scales, dlast)
    R.close(got["ddt"], *ref["ddt"], bf, "ddt")
    assert (ref["dA"][0] - (d * da).sum(0)).abs().max() <= 2.0 ** -40 * (d * dam).sum()


# ---- the convolution's ring -----------------------------------------------

@pytest.mark.parametrize("io,channels,total", [(bf, 1000, 12000), (f16, 4096, 6000), (f32, 67, 9000), (bf, 67, 70000)])
def test_conv_ring_of_sequences_that_start_anywhere(io, channels, total):
    """Continued sequences that start at every place of a run and of a
    workgroup's runs, in more workgroups than run at once, short runs and long
    ones, vectors and single channels: the tokens that see the ring see it as it
    was before the call."""
    log(f"[conv ring] {io} channels={channels} total={total}")
    g, lens = _gen(channels), []
    pick = torch.randint(0, 6, (total,), generator=g).tolist()
    while sum(lens) < total:
        lens.append((4, 5, 7, 13, 50, 121)[pick[len(lens)]])
    cu, nseq = R.sequences(lens), len(lens)
    T = cu[-1]
    x, w, b = _randn(g, T, channels, dtype=io), _randn(g, channels, 4, scale=0.5), _randn(g, channels)
    ring = _randn(g, nseq, channels, 4, dtype=io)
    seen = [3 + s % 9 for s in range(nseq)]
    assert {c % 48 for c in cu[:-1]} == set(range(48))
    # the tokens that see the ring, and some that do not
    near = sorted({c + k for c, n in zip(cu, lens) for k in range(min(n, 5))})
    at = torch.tensor(near)
    first, before = torch.zeros(T, dtype=torch.long), torch.zeros(nseq, 3, channels, dtype=R.f64)
    of = torch.zeros(T, dtype=torch.long)
    after = ring.clone()
    for s, n in enumerate(lens):
        first[cu[s]:cu[s + 1]], of[cu[s]:cu[s + 1]] = cu[s], s
        for j in range(3):
            before[s, j] = ring[s, :, (seen[s] - 3 + j) % 4].to(R.f64)
        for t in range(n - 4, n):
            after[s, :, (seen[s] + t) % 4] = x[cu[s] + t]
    pre, mag = b.to(R.f64).expand(len(near), channels).clone(), b.to(R.f64).abs().expand(len(near), channels).clone()
    for k in range(4):
        src = at - 3 + k
        inside = (src >= first[at])[:, None]
        v = torch.where(inside, x[src.clamp(min=0)].to(R.f64), before[of[at], (src - first[at] + 3).clamp(0, 2)])
        pre += v * w[:, k].to(R.f64)
        mag += (v * w[:, k].to(R.f64)).abs()
    ref = R.silu(pre)
    dx, dw, db, dcu, dseen = x.cuda(), w.cuda(), b.cuda(), _ints(cu), _ints(seen)
    for _ in range(3):
        dring = ring.cuda()
        out = binding.causal_conv1d_varlen_fwd(dx, dw, dcu, bias=db, activation="silu", conv_state=dring, cache_seqlens=dseen)
        R.close(out[at.cuda()], ref, 1.1 * mag, io, "out", R.SHORT)
        assert torch.equal(dring.cpu().view(torch.uint8), after.view(torch.uint8)), "ring"


@pytest.mark.parametrize("io,channels,total", [(bf, 64, 200), (f32, 67, 200), (bf, 4096, 3000), (bf, 67, 40000)])
@pytest.mark.parametrize("edge", [-3, -40])
def test_conv_edge_below_zero(io, channels, total, edge):
    """A first edge below 0 stands for 0, forward and backward, short runs and
    long ones.  (The rows before the tokens are there, and not read.)"""
    log(f"[conv edge] {io} channels={channels} total={total} edge={edge}")
    g = _gen(total)
    room = torch.full((total + 64, channels), float("nan"), dtype=io, device="cuda")
    x = room[64:]
    x.copy_(_randn(g, total, channels, dtype=io))
    w, dout = _randn(g, channels, 4, scale=0.5).cuda(), _randn(g, total, channels, dtype=io).cuda()
    got = []
    for first in (0, edge):
        cu = _ints([first, total // 2, total])
        got.append(binding.causal_conv1d_varlen_bwd(x, w, cu, dout, activation="silu"))
        got[-1]["out"] = binding.causal_conv1d_varlen_fwd(x, w, cu, activation="silu")
    for k in ("out", "dx", "dweight"):
        assert torch.equal(got[0][k], got[1][k]) and torch.isfinite(got[0][k]).all(), k


# ---- a stream of the caller's ---------------------------------------------

def _off(t):
    """The values of t at a place and with strides that make a wrapper copy them."""
    room = torch.empty(tuple(t.shape[:-1]) + (t.shape[-1] + 1,), dtype=t.dtype, device="cuda")
    room[..., 1:] = t
    return room[..., 1:]


def _busy(a, n=30):
    for _ in range(n):
        a = a @ a
    return a


def _packed_calls():
    """{name: call(stream) -> tensors} of the packed operators, on inputs that
    have to be copied first."""
    g, lens, h, G, n = _gen(21), (300, 1, 129), 4, 2, 64
    cu, T, ch = _ints(R.sequences(lens)), sum(lens), h * R.P + 2 * G * n
    x, B, C, dout = (_off(_randn(g, T, k, w, dtype=bf).cuda()) for k, w in ((h, R.P), (G, n), (G, n), (h, R.P)))
    dt, A = _off((_randn(g, T, h, dtype=bf) - 3).cuda()), _off(-1 - 7 * torch.rand(1, h, generator=g).cuda())[0]
    w, rows, drows = _off(_randn(g, ch, 4).cuda()), _off(_randn(g, T, ch, dtype=bf).cuda()), _off(_randn(g, T, ch, dtype=bf).cuda())
    rows_t = _randn(g, ch, T, dtype=bf).cuda().t()
    first = _off(_randn(g, len(lens), h, R.P, n).cuda())
    codes = torch.zeros(binding.ssd_checkpoint_slots(T, len(lens)), h, R.P, n, dtype=torch.int8, device="cuda")
    scales = torch.ones(codes.shape[:3], device="cuda")
    scan = (x, dt, A, B, C, cu, 300)
    binding.ssd_varlen_fwd(*scan, dt_softplus=True, checkpoints=(codes, scales))
    codes = _off(codes)

    ring, state = torch.ones(T, ch, 4, dtype=bf, device="cuda"), torch.ones(T, h, R.P, n, device="cuda")

    def step(stream):   # of new requests, which read neither cache
        out = binding.conv1d_ssd_update(rows_t, dt, A, w, ring, state, None, dt_softplus=True, stream=stream)
        return [out, ring, state]

    def grads(stream):
        got = binding.ssd_varlen_bwd(*scan, dout, (codes, scales), dt_softplus=True, dfinal_states=first, seq_segments=3,
                                     want_dinitial_states=True, stream=stream)
        return [got[k] for k in sorted(got)]

    def conv_grads(stream):
        got = binding.causal_conv1d_varlen_bwd(rows_t, w, cu, drows, activation="silu", stream=stream)
        return [got["dx"], got["dweight"]]

    return {"conv": lambda stream: [binding.causal_conv1d_varlen_fwd(rows_t, w, cu, stream=stream)], "conv_bwd": conv_grads,
            "scan": lambda stream: [binding.ssd_varlen_fwd(*scan, dt_softplus=True, seq_segments=3, stream=stream)],
            "scan_bwd": grads, "step": step}


def _check_stream(call):
    want = [v.clone() for v in call(None)]
    big, sizes = torch.randn(2048, 2048, device="cuda") / 64, [1 << k for k in range(9, 25)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    current = torch.cuda.current_stream()
    for busy_current in (True, False):
        if busy_current:   # a copy of an input left on the current stream would come long after the kernels
            _busy(big)
        else:              # the call's memory is still in use when it returns
            side.wait_stream(current)
            with torch.cuda.stream(side):
                _busy(big)
        got = call(side)
        assert torch.cuda.current_stream() == current
        junk = [torch.full((s,), float("nan"), device="cuda") for s in sizes for _ in range(3)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        del junk


@pytest.mark.parametrize("name", ["conv", "conv_bwd", "scan", "scan_bwd", "step"])
def test_explicit_stream(name):
    """stream= of another stream than the current one: inputs that are copied,
    workspaces and outputs all belong to it."""
    log(f"[stream] {name}")
    _check_stream(_packed_calls()[name])


def _dense_calls():
    """The same of the operators on dense rows."""
    g, b, d, l, n, h = _gen(22), 2, 128, 400, 16, 2
    r = lambda *shape, dtype=bf: _off(_randn(g, *shape, dtype=dtype).cuda())  # noqa: E731
    u, delta, dout, B, C = r(b, d, l), r(b, d, l) * 0.1, r(b, d, l), r(b, 1, n, l), r(b, 1, n, l)
    A = _off(-1 - torch.rand(d, n, generator=g).cuda())
    u, delta, dout = (v.transpose(1, 2).contiguous().transpose(1, 2) for v in (u, delta, dout))
    fwd = (u, delta, A, B, C)
    checkpoints = torch.zeros(b, d, binding.checkpoint_count(l), n, device="cuda")
    binding.ssm_scan_fwd(*fwd, delta_softplus=True, checkpoints=checkpoints)
    kept = _off(checkpoints)
    x, dt, Bs, Cs, As = r(b, l, h, R.P), r(b, l, h) - 3, r(b, l, 1, 64), r(b, l, 1, 64), -1 - torch.rand(h, generator=g).cuda()
    dt = _off(dt)
    w, bias = r(d, 4, dtype=f32), r(d, dtype=f32)
    start, xs = _randn(g, b, d, n).cuda(), r(b, d)

    def grads(stream):
        got = binding.ssm_scan_bwd(*fwd, dout, kept, delta_softplus=True, stream=stream)
        return [got[k] for k in sorted(got) if got[k] is not None]

    def update(stream):
        state = out_state   # refilled on the call's own stream
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            state.copy_(start)
        return [binding.selective_state_update(state, xs, xs, A, B[:, 0, :, 0], C[:, 0, :, 0], dt_softplus=True, stream=stream), state]

    out_state = torch.empty_like(start)
    return {"scan": lambda s: [binding.ssm_scan_fwd(*fwd, delta_softplus=True, seq_segments=3, stream=s)], "scan_bwd": grads,
            "conv": lambda s: [binding.causal_conv1d_fwd(u, w, bias, stream=s)],
            "conv_ex": lambda s: [binding.causal_conv1d_fwd_ex(u, w, bias, stream=s)],
            "ssd": lambda s: [binding.ssd_scan_fwd(x, dt, As, Bs, Cs, dt_softplus=True, seq_segments=3, stream=s)],
            "chunk_state": lambda s: list(binding.ssd_chunk_state(x, dt, As, Bs, 64, dt_softplus=True, stream=s)),
            "update": update}


@pytest.mark.parametrize("name", ["scan", "scan_bwd", "conv", "conv_ex", "ssd", "chunk_state", "update"])
def test_explicit_stream_of_dense_rows(name):
    log(f"[stream] dense rows: {name}")
    _check_stream(_dense_calls()[name])


# ---- decays after large steps ---------------------------------------------

def _large_steps(n, large, T=130, h=4):
    g = _gen(n)
    t = dict(x=_randn(g, T, h, R.P, dtype=bf), A=-8 - 5 * torch.rand(h, generator=g), B=_randn(g, T, 1, n, dtype=bf),
             C=_randn(g, T, 1, n, dtype=bf), dt=(0.004 + 0.008 * torch.rand(T, h, generator=g)).to(bf))
    for k in range(0, T, 16):
        t["dt"][k:k + 2] = large
    return t, [0, T]


@pytest.mark.parametrize("n", [32, 128])
@pytest.mark.parametrize("large", [1.0, 100.0, 3000.0])
def test_state_after_large_steps(n, large):
    """A chunk's running sum far from zero (to -3e5), and small steps after it:
    what remains of an input at the chunk's end is that of its own distance, to
    32 bits, and so are the gradients that the same decays carry."""
    log(f"[decay] state n={n} large={large}")
    t, cu = _large_steps(n, large)
    _, _, last, lastm, held = R.scan_fwd(t, cu)
    state = torch.empty(1, 4, R.P, n, device="cuda")
    binding.ssd_varlen_fwd(*(t[k].cuda() for k in ("x", "dt", "A", "B", "C")), _ints(cu), cu[-1], ssm_state=state)
    R.close(state, last, lastm, f32, "state")
    entries = binding.ssd_checkpoint_slots(cu[-1], 1)
    codes, scales = torch.zeros(entries, 4, R.P, n, dtype=torch.int8), torch.ones(entries, 4, R.P)
    for e, (S, _) in held.items():
        codes[e], scales[e] = R.to_8_bits(S.float())
    dout = _randn(_gen(n + 1), cu[-1], 4, R.P, dtype=bf)
    got, ref = _bwd(t, cu, dout, codes, scales, None), R.scan_bwd(t, cu, dout, codes, scales)
    for k in ("dx", "dB", "dC"):
        R.close(got[k], *ref[k], bf, k)
    da, dam = _through(t, cu, dout, codes, scales, None)
    d = t["dt"].to(R.f64)
    R.close(got["dA"], (d * da).sum(0), (d * dam).sum(0), f32, "dA")


@pytest.mark.parametrize("n", [32, 128])
@pytest.mark.parametrize("large", [1.0, 100.0, 3000.0])
def test_outputs_after_large_steps(n, large):
    """The same for the outputs, whose decays are between two tokens."""
    log(f"[decay] outputs n={n} large={large}")
    t, cu = _large_steps(n, large)
    ref, mag, *_ = R.scan_fwd(t, cu)
    out = binding.ssd_varlen_fwd(*(t[k].cuda() for k in ("x", "dt", "A", "B", "C")), _ints(cu), cu[-1])
    R.close(out, ref, mag, bf, "out")


# ---- dense inputs at any address ------------------------------------------

def _shifted(t):
    """t, dense, four bytes behind a 16-byte address."""
    room = torch.empty(t.numel() + 1, dtype=f32, device="cuda")
    v = room[1:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16 == 4
    return v


def test_parameters_at_any_address():
    """Weights and gradients that lie in one flat buffer, as a sharded optimiser
    keeps them."""
    log("[address]")
    g, h, n, b = _gen(2), 3, 32, 5
    ch = h * R.P + 2 * n
    xbc, dt, A = _randn(g, b, ch, dtype=bf).cuda(), _randn(g, b, h, dtype=bf).cuda(), -1 - torch.rand(h, generator=g).cuda()
    w, bias = _randn(g, ch, 4).cuda(), _randn(g, ch).cuda()
    outs = []
    for wk, bk in ((w, bias), (_shifted(w), _shifted(bias))):
        ring, state = torch.zeros(b, ch, 4, dtype=bf, device="cuda"), torch.zeros(b, h, R.P, n, device="cuda")
        outs.append((binding.conv1d_ssd_update(xbc, dt, A, wk, ring, state, None, conv_bias=bk, dt_softplus=True), state))
        outs[-1] += (binding.causal_conv1d_varlen_fwd(xbc, wk, _ints([0, b]), bias=bk),)
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    t, cu, dout, codes, scales, dlast = _steps_case(1, (70, 3), 2, 1, 32, 1.0)
    want = _bwd(t, cu, dout, codes, scales, dlast)
    got = binding.ssd_varlen_bwd(*(t[k].cuda() for k in ("x", "dt", "A", "B", "C")), _ints(cu), 70, dout.cuda(),
                                 (codes.cuda(), scales.cuda()), dfinal_states=_shifted(dlast.cuda()))
    assert all(torch.equal(want[k], got[k]) for k in want)


@pytest.mark.parametrize("lens,n,G,decay", [((94,) * 12, 32, 4, 0.05), ((700,), 128, 1, 0.01), ((130, 70, 200), 64, 2, 0.02)])
def test_decay_gradient_to_32_bits(lens, n, G, decay):
    """dA against 64 bits, over all heads.  Every path's factors have 24 bits and
    take some eight roundings of 2^-24 (products, decays, partial sums), and the
    paths have any sign, as their roundings do: sqrt(8) 2^-24 of the whole, 2^-21
    with what the draw can add.  Inputs with a mean, so that roundings to one
    side would add up."""
    log(f"[decay] 32 bits lens={lens} n={n}")
    h = 16
    t, cu, dout, codes, scales, _ = _steps_case(n, lens, h, G, n, decay)
    for k in ("x", "B", "C"):
        t[k] = R.silu(t[k].float()).to(bf)
    for e, (S, _) in R.scan_fwd(t, cu)[4].items():
        codes[e], scales[e] = R.to_8_bits(S.float())
    da, _ = _through(t, cu, dout, codes, scales, None)
    ref = (t["dt"].to(R.f64) * da).sum(0)
    got = _bwd(t, cu, dout, codes, scales, None)["dA"].cpu().to(R.f64)
    off = ((got - ref).norm() / ref.norm()).item()
    log(f"  relative error {off:.2e}")
    assert off <= 2.0 ** -21


@pytest.mark.parametrize("single", [False, True])
def test_steps_to_32_bits(single):
    """softplus(dt + bias) from a state that one token leaves, dt' x B with x and B
    of 1: exp2, log2 and reciprocal of the hardware are off by 2^-23 each, and six
    operations round by 2^-24: below 2^-21, at steps down to 1e-6."""
    log(f"[steps] single={single}")
    g, T, h, n = _gen(1), 400, 64, 32
    dt, bias = (3 * torch.randn(T, h, generator=g) - 3).to(bf), -2 - 4 * torch.rand(h, generator=g)
    A, state = -torch.ones(h), torch.empty(T, h, R.P, n, device="cuda")
    if single:
        xbc = torch.ones(T, h * R.P + 2 * n, dtype=bf, device="cuda")
        w = torch.zeros(h * R.P + 2 * n, 4, device="cuda")
        w[:, 3] = 1
        ring = torch.zeros(T, h * R.P + 2 * n, 4, dtype=bf, device="cuda")
        binding.conv1d_ssd_update(xbc, dt.cuda(), A.cuda(), w, ring, state, None, dt_bias=bias.cuda(), dt_softplus=True,
                                  activation=None)
    else:
        one = torch.ones(T, h, R.P, dtype=bf, device="cuda")
        B = torch.ones(T, 1, n, dtype=bf, device="cuda")
        binding.ssd_varlen_fwd(one, dt.cuda(), A.cuda(), B, B, torch.arange(T + 1, dtype=i32, device="cuda"), 1,
                               dt_bias=bias.cuda(), dt_softplus=True, ssm_state=state)
    v = (dt.float() + bias).to(R.f64)   # the sum is rounded to 32 bits, as a token's own logit
    ref = torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)
    off = ((state[:, :, 5, 7].cpu().to(R.f64) - ref) / ref).abs().max().item()
    log(f"  relative error {off:.2e}")
    assert ref.min() < 2e-6 and off <= 2.0 ** -21


# ---- values that are not finite -------------------------------------------

@pytest.mark.parametrize("n", [32, 128])
@pytest.mark.parametrize("which", ["x", "B", "C", "dt", "dout"])
def test_scan_keeps_to_its_sequence(which, n):
    """Infinities and NaN of one sequence reach no token and no state of another,
    forward or backward, whatever lies in the same 64 tokens of memory."""
    log(f"[not finite] {which} n={n}")
    lens, h = (70, 30, 3, 100), 4
    t, cu, dout, codes, scales, _ = _steps_case(n, lens, h, 2, n, 1.0)
    runs = []
    for bad in (False, True):
        v = {k: u.clone() for k, u in dict(t, dout=dout).items()}
        if bad:
            part = v[which][cu[1]:cu[2]]
            part[3::7], part[5::7] = float("nan"), float("inf")
        state = torch.empty(4, h, R.P, n, device="cuda")
        out = binding.ssd_varlen_fwd(*(v[k].cuda() for k in ("x", "dt", "A", "B", "C")), _ints(cu), 100, ssm_state=state)
        runs.append((out, state, _bwd(v, cu, v["dout"], codes, scales, None)))
    others = torch.ones(cu[-1], dtype=torch.bool)
    others[cu[1]:cu[2]] = False
    others = others.cuda()
    (a, sa, ga), (b, sb, gb) = runs
    assert torch.equal(a[others], b[others]) and torch.equal(sa[[0, 2, 3]], sb[[0, 2, 3]])
    for k in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(ga[k][others], gb[k][others]), k
    assert not all(torch.isfinite(gb[k].float()).all() for k in ("dx", "ddt", "dB", "dC"))


@pytest.mark.parametrize("n", [32, 128])
def test_values_that_are_not_finite_inside_a_sequence(n):
    """In the forward a B, C or dt that is not finite reaches no token before its
    own, and an x no other channel and none of the tokens before its block of 32;
    its own and later ones are not finite either."""
    log(f"[not finite] inside n={n}")
    t, cu, *_ = _steps_case(n, (130,), 4, 2, n, 1.0)
    at = 64 + 40
    for which in ("x", "B", "C", "dt"):
        outs = []
        for bad in (False, True):
            v = {k: u.clone() for k, u in t.items()}
            if bad:
                (v["x"][at, 1, 9:10] if which == "x" else v[which][at]).fill_(float("nan"))
            outs.append(binding.ssd_varlen_fwd(*(v[k].cuda() for k in ("x", "dt", "A", "B", "C")), _ints(cu), 130).cpu())
        a, b = outs
        if which == "x":
            rest = torch.ones(4, R.P, dtype=torch.bool)
            rest[1, 9] = False
            assert torch.equal(a[:, rest], b[:, rest]) and torch.equal(a[:at // 32 * 32], b[:at // 32 * 32])
            assert torch.isnan(b[at:, 1, 9]).all()
        else:
            assert torch.equal(a[:at], b[:at]) and torch.isnan(b[at]).all(), which
            assert which == "C" or torch.isnan(b[at:]).all(), which


@pytest.mark.parametrize("decay", [0.0, 0.003, 0.05])
def test_states_to_32_bits(decay):
    """The last state against 64 bits, over all its elements, after many chunks
    whose terms have a mean.  A term has the roundings of its step's decay (exp2
    and four operations) and of its products: sqrt(6) 2^-24 / sqrt(3) if they fall
    as they may; the sums' add one of each chunk's nine, as partial sums are as
    large as the state.  Together sqrt(6 + 9) 2^-24 / sqrt(3) = 1.3e-7, here with
    steps that are given and one segment: 2^-23."""
    log(f"[state] decay={decay}")
    g, T, h, n = _gen(7), 1500, 3, 128
    t = dict(x=R.silu(_randn(g, T, h, R.P)).to(bf), A=-decay * (0.5 + torch.rand(h, generator=g)),
             B=R.silu(_randn(g, T, 1, n)).to(bf), C=_randn(g, T, 1, n, dtype=bf), dt=(0.75 + 0.5 * torch.rand(T, h, generator=g)).to(bf))
    last = R.scan_fwd(t, [0, T])[2]
    state = torch.empty(1, h, R.P, n, device="cuda")
    binding.ssd_varlen_fwd(*(t[k].cuda() for k in ("x", "dt", "A", "B", "C")), _ints([0, T]), T, ssm_state=state, seq_segments=1)
    off = ((state.cpu().to(R.f64) - last).norm() / last.norm()).item()
    log(f"  relative error {off:.2e}")
    assert off <= 2.0 ** -23
