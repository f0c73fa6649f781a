"""The gated block's operators as they are used: together, on streams of the
caller's, in captured graphs, at far offsets, and by several callers at once."""
import importlib.util
import os

import pytest
import torch

from state_space_model_scan_amd import binding
from tests import gated_ref as R
from tests.harness import log
from tests.test_gpu_varlen_edges import _check_stream, _off

pytestmark = pytest.mark.gpu
bf, f16, f32, i32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


def _ints(v):
    return torch.tensor(v, dtype=i32, device="cuda")


def _rand(seed, *shape, dtype=f32, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def _scan_inputs(T, C, seed=0, io=bf):
    x, r, i, dout = (_rand(seed + k, T, C, dtype=io) for k in range(4))
    A, rb, ib = -torch.rand(C, generator=torch.Generator().manual_seed(seed + 9)).cuda(), _rand(seed + 5, C), _rand(seed + 6, C)
    return (x, r, i, A), dict(r_bias=rb, i_bias=ib), dout


def _calls():
    """{name: call(stream) -> tensors}, on inputs that have to be copied first."""
    lens, C = (300, 0, 1, 129), 72
    cu, T = _ints(R.sequences(lens)), sum(lens)
    (x, r, i, A), kw, dout = _scan_inputs(T, C)
    t = lambda v: v.t().contiguous().t()  # noqa: E731  (a token's channels apart: copied)
    kept = torch.empty(-(-T // 64), C, device="cuda")
    binding.gated_scan_varlen_fwd(x, r, i, A, cu, checkpoints=kept, **kw)
    A, kw = _off(A[None])[0], {k: torch.stack([v, v], 1)[:, 0] for k, v in kw.items()}
    args, dout, kept, first = (t(x), t(r), t(i), A, torch.stack([cu, cu], 1)[:, 0]), t(dout), t(kept), t(_rand(3, 4, C))
    state = torch.ones(T, C, device="cuda")

    def grads(stream):
        got = binding.gated_scan_varlen_bwd(*args, dout, kept, dfinal_states=first, want_dinitial_states=True, stream=stream, **kw)
        return [got[k] for k in sorted(got)]

    def step(stream):   # of new requests
        return [binding.gated_scan_update(*args[:4], state, None, stream=stream, **kw), state]

    nx, nw, res, z, dy = t(_rand(1, 300, 520, dtype=bf)), torch.stack([_rand(2, 520)] * 2, 1)[:, 0], t(_rand(4, 300, 520)), \
        t(_rand(5, 300, 520, dtype=bf)), t(_rand(6, 300, 520, dtype=bf))

    def norm_grads(stream):
        got = binding.rms_norm_bwd(res, nw, dy, ds=res, stream=stream)
        return [got[k] for k in sorted(got)]

    return {"scan": lambda s: [binding.gated_scan_varlen_fwd(*args, stream=s, **kw)], "scan_bwd": grads, "step": step,
            "norm": lambda s: list(binding.rms_norm_fwd(nx, nw, residual=res, stream=s)),
            "gated norm": lambda s: [binding.rms_norm_fwd(nx, nw, z=z, group_size=104, stream=s)],
            "norm to 8 bits": lambda s: [v.view(torch.uint8) for v in binding.rms_norm_quant_fwd(nx, nw, residual=res, stream=s)],
            "norm_bwd": norm_grads}


@pytest.mark.parametrize("name", ["scan", "scan_bwd", "step", "norm", "gated norm", "norm to 8 bits", "norm_bwd"])
def test_explicit_stream(name):
    log(f"[gated stream] {name}")
    _check_stream(_calls()[name])


def _training_step(C=200, lens=(200, 1, 63, 0, 300), seed=0):
    """A function that runs norm, scan and their gradients once, and its results."""
    cu, T = _ints(R.sequences(lens)), sum(lens)
    (_, r, i, A), kw, dout = _scan_inputs(T, C, seed)
    res, w, dy = _rand(seed + 20, T, C), _rand(seed + 21, C), _rand(seed + 22, T, C, dtype=bf)
    branch = _rand(seed + 23, T, C, dtype=bf)
    kept = torch.empty(-(-T // 64), C, device="cuda")

    def step():
        x, stream = binding.rms_norm_fwd(branch, w, residual=res)
        h = binding.gated_scan_varlen_fwd(x, r, i, A, cu, checkpoints=kept, **kw)
        y = binding.rms_norm_fwd(h, w, z=r, group_size=C // 5)
        codes, scales = binding.rms_norm_quant_fwd(h, w)
        n = binding.rms_norm_bwd(h, w, dy, z=r, group_size=C // 5)
        g = binding.gated_scan_varlen_bwd(x, r, i, A, cu, n["dx"], kept, **kw)
        f = binding.rms_norm_bwd(stream, w, g["dx"], ds=res)
        return [x, stream, h, y, codes.view(torch.uint8), scales, kept] + [d[k] for d in (n, g, f) for k in sorted(d)]

    return step


def test_captured_training_step():
    """In a graph, replayed between eager calls and synchronisations."""
    step = _training_step()
    want = [v.clone() for v in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        for a, b in zip(want, step()):
            assert torch.equal(a, b)


def test_two_graphs_of_one_workspace():
    """Two captured calls that are given the same workspace, replayed in turn, and
    eager calls with it between them; the workspace holds what others left."""
    C, lens = 130, (700, 3, 400)
    cu, T = _ints(R.sequences(lens)), sum(lens)
    ws = torch.full((1 << 22,), 0x5a, dtype=torch.uint8, device="cuda")
    runs = []
    for seed in (0, 50):
        args, kw, dout = _scan_inputs(T, C, seed)
        kept = torch.empty(-(-T // 64), C, device="cuda")

        def run(args=args, kw=kw, dout=dout, kept=kept):
            out = binding.gated_scan_varlen_fwd(*args, cu, checkpoints=kept, workspace=ws, **kw)
            g = binding.gated_scan_varlen_bwd(*args, cu, dout, kept, workspace=ws, **kw)
            return [out] + [g[k] for k in sorted(g)]

        want = [v.clone() for v in run()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        runs.append((run, want, graph, got))
    for k in range(3):
        ws.fill_(0xff if k == 1 else 0)
        for run, want, graph, got in runs:
            for v in got:
                v.zero_()
            graph.replay()
            for a, b in zip(want, got):
                assert torch.equal(a, b)
            for a, b in zip(want, run()):
                assert torch.equal(a, b)


def test_calls_at_once():
    """Several calls in flight on streams of their own: their tiles wait for each
    other in the same compute units."""
    log("[gated] at once")
    runs = [_training_step(C, lens, seed) for C, lens, seed in ((900, (3000, 5, 1200), 1), (520, (6000,), 2), (1100, (64,) * 40, 3))]
    want = [[v.clone() for v in run()] for run in runs]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        got = []
        for run, s in zip(runs, side):
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_a_small_workspace_is_refused():
    args, kw, dout = _scan_inputs(300, 64)
    cu, kept, ws = _ints([0, 300]), torch.empty(5, 64, device="cuda"), torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        binding.gated_scan_varlen_fwd(*args, cu, workspace=ws, **kw)
    with pytest.raises(ValueError, match="workspace"):
        binding.gated_scan_varlen_bwd(*args, cu, dout, kept, workspace=ws, **kw)
    with pytest.raises(ValueError, match="workspace"):
        binding.rms_norm_bwd(_rand(0, 3000, 64), _rand(1, 64), _rand(2, 3000, 64), workspace=ws)
    with pytest.raises(ValueError, match="workspace"):
        binding.gated_scan_varlen_fwd(*args, cu, workspace=torch.empty(1 << 20, dtype=torch.uint8), **kw)


def test_offsets_past_32_bits():
    """Tokens, rows and cache entries whose byte offsets pass 2^32."""
    log("[gated] far")
    C, T, far = 64, 150, 1 << 24
    (x, r, i, A), kw, _ = _scan_inputs(T, C)
    cu = _ints([0, 70, T])
    want = binding.gated_scan_varlen_fwd(x, r, i, A, cu, **kw)
    room = torch.empty((T - 1) * far + C, dtype=bf, device="cuda")   # 5 GB
    wide = room.as_strided((T, C), (far, 1))
    wide.copy_(x)
    assert torch.equal(want, binding.gated_scan_varlen_fwd(wide, r, i, A, cu, **kw))
    out = binding.gated_scan_varlen_fwd(x, r, i, A, cu, out=wide, **kw)
    assert torch.equal(out, want)
    w = _rand(4, C)
    normed = binding.rms_norm_fwd(x, w)
    wide.copy_(x)
    assert torch.equal(normed, binding.rms_norm_fwd(wide, w))
    assert torch.equal(binding.rms_norm_fwd(x, w, out=wide), normed)
    with pytest.raises(ValueError):   # rows too far apart for the recurrence's offsets
        binding.gated_scan_varlen_fwd(room.as_strided((20, C), (far + 1, 1)), r[:20], i[:20], A, _ints([0, 20]), **kw)
    del room, wide, out
    entries = (1 << 31) // C + 3
    state = torch.empty(entries, C, device="cuda")   # 8.6 GB
    state[-1] = 1.0
    for slots in (None, _ints([entries - 1, -1])):
        cache = torch.ones(2, C, device="cuda")
        near = binding.gated_scan_varlen_fwd(x, r, i, A, cu, state=cache, cache_seqlens=_ints([1, 1]), slots=_ints([0, -1]), **kw)
        if slots is None:
            continue
        got = binding.gated_scan_varlen_fwd(x, r, i, A, cu, state=state, cache_seqlens=_ints([1, 1]), slots=slots, **kw)
        assert torch.equal(near, got) and torch.equal(state[-1], cache[0])


def test_broadcast_inputs():
    """Inputs of one row for all tokens, and one tensor for several arguments."""
    (x, r, i, A), kw, dout = _scan_inputs(100, 40)
    cu = _ints([0, 60, 100])
    one = r[:1].expand(100, 40)
    assert torch.equal(binding.gated_scan_varlen_fwd(x, one, one, A, cu, **kw),
                       binding.gated_scan_varlen_fwd(x, one.contiguous(), one.contiguous(), A, cu, **kw))
    a, b = binding.gated_scan_varlen_fwd(x, x, x, A, cu), binding.gated_scan_varlen_fwd(x, x.clone(), x.clone(), A, cu)
    assert torch.equal(a, b)
    w = torch.ones(1, device="cuda").expand(40)
    assert torch.equal(binding.rms_norm_fwd(one, w), binding.rms_norm_fwd(one.contiguous(), w.contiguous()))
    assert torch.equal(binding.rms_norm_fwd(x, w, z=x), binding.rms_norm_fwd(x, w.contiguous(), z=x.clone()))
    got, want = binding.rms_norm_bwd(x, w, x, ds=x), binding.rms_norm_bwd(x, w.contiguous(), x.clone(), ds=x.clone())
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("cu", [[5, 3, 70, 20, 100], [-4, 30, 260, 90, 100], [100, 0, 0, 0, 0], [0, 0, 0, 0, 2 ** 31 - 1]])
def test_edges_out_of_order_stay_inside(cu):
    """Edges that are no edges: unspecified results, but nothing outside the
    tensors is touched and every call ends."""
    T, C = 100, 40
    room = torch.full((T + 2, C), 9.0, dtype=bf, device="cuda")
    (x, r, i, A), kw, dout = _scan_inputs(T, C)
    caches = torch.full((6, C), 9.0, device="cuda")
    binding.gated_scan_varlen_fwd(x, r, i, A, _ints(cu), out=room[1:-1], state=caches[1:-1], **kw)
    grads = torch.full((3, T + 2, C), 9.0, dtype=bf, device="cuda")
    binding.gated_scan_varlen_bwd(x, r, i, A, _ints(cu), dout, torch.zeros(2, C, device="cuda"), dx=grads[0, 1:-1],
                                  dr=grads[1, 1:-1], di=grads[2, 1:-1], want_dinitial_states=True, **kw)
    torch.cuda.synchronize()
    assert (room[[0, -1]] == 9).all() and (caches[[0, -1]] == 9).all() and (grads[:, [0, -1]] == 9).all()


# ---- the example ------------------------------------------------------------

def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")
    spec = importlib.util.spec_from_file_location("gated_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def _plain_block(w, group, branch, stream, lens):
    """The example's block in 64 bits on the CPU, for torch's own differentiation."""
    def norm(v, weight, n):
        by = v.view(v.shape[0], -1, n)
        return (by / torch.sqrt((by * by).mean(-1, keepdim=True) + 1e-5)).view_as(v) * weight

    inner = w["A"].shape[0]
    held = branch + stream
    row = norm(held, w["norm"], held.shape[1]) @ w["w_in"].t()
    z, x = row[:, :inner], row[:, inner:]
    us, hs = [], []
    for part in x.split(list(lens)):
        v = torch.cat([part.new_zeros(3, inner), part])
        us.append(w["conv_bias"] + sum(v[k:k + part.shape[0]] * w["conv"][:, k] for k in range(4)))
    u = torch.cat(us)
    gates = u @ w["w_gates"].t()
    a = torch.exp(w["A"] * torch.sigmoid(gates[:, :inner] + w["r_bias"]))
    b = torch.sqrt(1 - a * a) * torch.sigmoid(gates[:, inner:] + w["i_bias"]) * u
    for pa, pb in zip(a.split(list(lens)), b.split(list(lens))):
        h = pa.new_zeros(inner)
        for k in range(pa.shape[0]):
            h = pa[k] * h + pb[k]
            hs.append(h)
    out = norm(torch.stack(hs) * z * torch.sigmoid(z), w["gated_norm"], group)
    return out @ w["w_out"].t(), held


def test_example_gradients():
    """Every gradient of the example's block against torch's differentiation of the
    plain one.  The branch's activations and products are in bf16, off by 2^-9 of
    their size on average: some twelve of them lie between a weight and the loss,
    whose squares add to (2^-9)^2 12, and as many on the way back; three times that
    is allowed, 3 sqrt(24) 2^-9."""
    ex = _example()
    block, lens = ex.Block(width=64, inner=96, groups=2), (50, 1, 67, 14)
    branch, stream, target = ex.data(lens, 64, 3)
    branch, cu = branch.bfloat16(), ex.packed(lens)
    out, held, saved = block.forward(branch, stream, cu)
    dbranch, dstream = target.bfloat16(), stream.clone()
    grads, dx, ds = block.backward(dbranch, dstream, saved, cu)
    w = {k: v.double().cpu().requires_grad_() for k, v in block.w.items()}
    b, s = branch.double().cpu().requires_grad_(), stream.double().cpu().requires_grad_()
    o, r = _plain_block(w, block.group, b, s, lens)
    ((o * dbranch.double().cpu()).sum() + (r * dstream.double().cpu()).sum()).backward()

    def off(got, want):
        return ((got.double().cpu() - want).norm() / want.norm()).item()

    far = {k: off(v, w[k].grad) for k, v in grads.items()}
    far.update(out=off(out, o.detach()), stream=off(held, r.detach()), dx=off(dx, b.grad), ds=off(ds, s.grad))
    log("[gated example] " + " ".join(f"{k} {v:.1e}" for k, v in far.items()))
    assert set(grads) == set(block.w)
    for k, v in far.items():
        assert v <= 3 * 24 ** 0.5 * 2.0 ** -9, (k, v)


def test_example_runs():
    ex = _example()
    block = ex.Block()
    losses = ex.train(block, steps=5)
    assert all(torch.isfinite(torch.tensor(losses)))
    got, want = ex.serve(block)
    # bf16 activations on both ways; a product of few rows may be summed in another order: a few roundings of 2^-8
    assert (got.float() - want.float()).norm() <= 8 * 2.0 ** -8 * want.float().norm()
