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


# ---- channels that grow -----------------------------------------------------

@pytest.mark.parametrize("io", [f32, bf])
@pytest.mark.parametrize("T,C", [(700, 72), (4200, 1030)])
def test_a_growing_channel_of_nothing_stays_nothing(io, T, C):
    """A > 0: an input weighs nothing, so from no state all of it is 0, though the
    decay of a tile's tokens overflows; and the others are what they are."""
    log(f"[gated growing] {io} {T}x{C}")
    g = torch.Generator().manual_seed(T)
    t = dict(x=_randn(g, T, C, dtype=io), r=_randn(g, T, C, dtype=io), i=_randn(g, T, C, dtype=io),
             A=-(0.05 + 3 * torch.rand(C, generator=g)))
    t["A"][::3] = 2.0
    rest = [c for c in range(C) if c % 3][:40]
    cu = [0, 5, T - 9, T]
    dout = _randn(g, T, C, dtype=io)
    dout[30:] = 0
    args = [t[k].cuda() for k in ("x", "r", "i", "A")]
    kept, state = torch.empty(-(-T // 64), C, device="cuda"), torch.zeros(3, C, device="cuda")
    out = binding.gated_scan_varlen_fwd(*args, _ints(cu), state=state, cache_seqlens=_ints([1] * 3), checkpoints=kept)
    assert not out[:, ::3].any() and not state[:, ::3].any() and not kept[:, ::3].any()
    grads = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept)
    for k, v in grads.items():
        assert not v[..., ::3].any(), k
    few = {k: v[..., rest] for k, v in t.items()}
    ref = R.scan(few, cu)
    R.close(out[:, rest], ref["after"], ref["err"], io, "out")
    want = R.scan_bwd(few, cu, dout[:, rest])
    for k, v in grads.items():
        R.close(v[..., rest], *want[k], io if k in ("dx", "dr", "di") else f32, k)


# ---- gates far open and far closed ------------------------------------------

@pytest.mark.parametrize("io,T,C", [(f32, 1, 40), (f32, 130, 256), (f32, 1700, 200), (f32, 3200, 4096), (bf, 3200, 4096),
                                    (f16, 3200, 4096), (bf, 500, 72)])
def test_gradients_of_open_gates(io, T, C):
    """dr and di carry 1 - sigma of a gate, to a relative bound: with
    w = exp(-v), sigma = 1 / (1 + w) and 1 - sigma = w sigma, w is off by
    (3 |v| + 2) u, sigma by (3 |v| + 5) u, the product by one rounding.  Sequences
    of a single token, so that every element stands by itself."""
    log(f"[gated open gates] {io} {T}x{C}")
    g = torch.Generator().manual_seed(T + C)

    def far():
        v = 8 + 12 * torch.rand(T, C, generator=g)
        return torch.where(torch.rand(T, C, generator=g) < 0.8, v, -v).to(io)

    t = dict(x=_randn(g, T, C, dtype=io), r=far(), i=far(), A=-(0.05 + 3 * torch.rand(C, generator=g)),
             r_bias=_randn(g, C, scale=0.25), i_bias=_randn(g, C, scale=0.25))
    dout = _randn(g, T, C, dtype=io)
    args, kw = [t[k].cuda() for k in ("x", "r", "i", "A")], {k: t[k].cuda() for k in ("r_bias", "i_bias")}
    cu = _ints(list(range(T + 1)))
    kept = torch.zeros(-(-T // 64), C, device="cuda")
    got = binding.gated_scan_varlen_bwd(*args, cu, dout.cuda(), kept, **kw)
    cols = sorted(set(range(min(C, 40))) | set(range(C - 8, C)))
    few = {k: v[..., cols] for k, v in t.items()}
    flat = {k: v.reshape(1, -1) if v.dim() == 2 else v.repeat(T) for k, v in few.items()}
    ref = R.scan_bwd(flat, [0, 1], dout[:, cols].reshape(1, -1))
    A, x = flat["A"].double(), flat["x"].double()

    def open_error(v, bias):   # of 1 - sigma, relative
        return R.U * (6 * (v.double() + bias.double()).abs() + 8)

    (q, e_q), (dx, e_dx) = ref["dA"], ref["dx"]
    for name, gate, e_rest in (("dr", "r", A.abs() * e_q), ("di", "i", e_dx * x.abs())):
        v = flat[gate].double() + flat[gate + "_bias"].double()
        closed = torch.sigmoid(-v)
        want = (A * q if name == "dr" else dx * x) * closed
        err = e_rest * closed + want.abs() * (open_error(flat[gate], flat[gate + "_bias"]) + 4 * R.U)
        want, err = want.view(T, -1), err.view(T, -1)
        R.close(got[name][:, cols], want, err, io, name)
        R.close(got[name + "_bias"][cols], want.sum(0), err.sum(0) + 130 * R.U * want.abs().sum(0), f32, name + "_bias")


# ---- the kernels of large 16-bit calls --------------------------------------

# (T, C, nseq): two channels a lane in the forward and 16 tokens a lane in the gradient, with fewer and with more
# sequences than a wave has lanes; large workgroups of few strips; odd widths
LARGE = [(4200, 3200, 150), (4200, 3200, 5), (4200, 1030, 5), (3100, 4097, 3), (1700, 200, 3), (130, 1000, 2)]


@pytest.mark.parametrize("io", [f16, bf])
@pytest.mark.parametrize("T,C,nseq", LARGE)
def test_large_16_bit_calls(io, T, C, nseq):
    log(f"[gated large] {io} {T}x{C} in {nseq}")
    g = torch.Generator().manual_seed(T + C + nseq)
    t = dict(x=_randn(g, T, C, dtype=io), r=_randn(g, T, C, dtype=io), i=_randn(g, T, C, dtype=io),
             A=-(0.05 + 3 * torch.rand(C, generator=g)), r_bias=_randn(g, C, scale=0.5), i_bias=_randn(g, C, scale=0.5))
    cu = [0] + sorted(torch.randint(0, T + 1, (nseq - 1,), generator=g).tolist()) + [T]
    dout, state, dfin = _randn(g, T, C, dtype=io), _randn(g, nseq, C), _randn(g, nseq, C)
    slots = torch.randperm(nseq, generator=g).tolist()
    args, kw = [t[k].cuda() for k in ("x", "r", "i", "A")], {k: t[k].cuda() for k in ("r_bias", "i_bias")}
    kept, dstate = torch.empty(-(-T // 64), C, device="cuda"), state.cuda()
    out = binding.gated_scan_varlen_fwd(*args, _ints(cu), state=dstate, cache_seqlens=_ints([1] * nseq), slots=_ints(slots),
                                        checkpoints=kept, **kw)
    got = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, initial_states=state[slots].cuda(),
                                        dfinal_states=dfin.cuda(), want_dinitial_states=True, **kw)
    # channels are independent: some of every strip's
    cols = sorted(set(range(0, C, 61)) | set(range(min(C, 4))) | set(range(C - 4, C)))
    few = {k: v[..., cols] for k, v in t.items()}
    ref, err, after, e_after = R.scan_cached(few, cu, state[:, cols], [1] * nseq, slots)
    R.close(out[:, cols], ref, err, io, "out")
    R.close(dstate[:, cols], after, e_after, f32, "cache")
    want = R.scan_bwd(few, cu, dout[:, cols], state[slots][:, cols], dfin[:, cols])
    for k, v in got.items():
        R.close(v[..., cols], *want[k], io if k in ("dx", "dr", "di") else f32, k)


# ---- far rows ---------------------------------------------------------------

def test_rows_far_apart():
    """Token and row strides of 2^24 elements, the largest that the scans take, in
    every operator that reads or writes such rows."""
    log("[gated far rows]")
    C, T, far = 64, 140, 1 << 24
    g = torch.Generator().manual_seed(2)
    room = torch.empty((T - 1) * far + 4 * C, dtype=bf, device="cuda")   # 4.7 GB

    def view(k):
        return room.as_strided((T, C), (far, 1), k * C)

    x, r, i, dout = (_randn(g, T, C, dtype=bf).cuda() for _ in range(4))
    A, cu, w = -torch.rand(C, generator=g).cuda(), _ints([0, 70, T]), _randn(g, C).cuda()
    kept = torch.empty(-(-T // 64), C, device="cuda")
    out = binding.gated_scan_varlen_fwd(x, r, i, A, cu, checkpoints=kept)
    want = binding.gated_scan_varlen_bwd(x, r, i, A, cu, dout, kept)
    for k, v in enumerate((x, r, i, dout)):
        view(k).copy_(v)
    got = binding.gated_scan_varlen_bwd(view(0), view(1), view(2), A, cu, view(3), kept)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    got = binding.gated_scan_varlen_bwd(x, r, i, A, cu, dout, kept, dx=view(0), dr=view(1), di=view(2))
    for k in want:
        assert torch.equal(want[k], got[k]), f"{k} into far rows"
    # the norm's gradient, and its 8 bits
    want = binding.rms_norm_bwd(x, w, dout, z=r)
    for k, v in enumerate((x, dout, r)):
        view(k).copy_(v)
    got = binding.rms_norm_bwd(view(0), w, view(1), z=view(2), dx=view(3))
    for k in want:
        assert torch.equal(want[k], got[k]), f"norm's {k}"
    got = binding.rms_norm_bwd(x, w, dout, z=r, dz=view(3))
    assert torch.equal(want["dz"], got["dz"])
    codes, scales = binding.rms_norm_quant_fwd(x, w, z=r)
    bytes_ = room.view(torch.float8_e4m3fn).as_strided((T, C), (2 * far, 1), 0)
    far_codes, far_scales = binding.rms_norm_quant_fwd(x, w, z=r, codes=bytes_)
    assert torch.equal(codes.view(torch.uint8), far_codes.contiguous().view(torch.uint8)) and torch.equal(scales, far_scales)
    # the step on rows far apart
    state = torch.ones(T, C, device="cuda")
    want = binding.gated_scan_update(x, r, i, A, state.clone(), None)
    view(0).copy_(x)
    assert torch.equal(want, binding.gated_scan_update(view(0), r, i, A, state.clone(), None, out=view(1)))
    del room
    # fp32, whose last token of a wave is 15 2^26 bytes from its first
    room = torch.empty((T // 2 - 1) * far + C, device="cuda").as_strided((T // 2, C), (far, 1))
    x, r, i, cu = x.float()[:T // 2], r.float()[:T // 2], i.float()[:T // 2], _ints([0, 3, T // 2])
    want = binding.gated_scan_varlen_fwd(x, r, i, A, cu)
    room.copy_(x)
    assert torch.equal(want, binding.gated_scan_varlen_fwd(room, r, i, A, cu))
    assert torch.equal(want, binding.gated_scan_varlen_fwd(x, r, i, A, cu, out=room))


def test_step_on_a_far_entry():
    """A cache entry whose byte offset passes 2^33, in the step."""
    log("[gated far entry]")
    C = 64
    g = torch.Generator().manual_seed(3)
    x, r, i = (_randn(g, 2, C, dtype=bf).cuda() for _ in range(3))
    A, entries = -torch.rand(C, generator=g).cuda(), (1 << 31) // C + 3
    state = torch.empty(entries, C, device="cuda")   # 8.6 GB
    state[-1] = 0.5
    near = torch.full((1, C), 0.5, device="cuda")
    want = binding.gated_scan_update(x, r, i, A, near, _ints([1, 1]), slots=_ints([0, -1]))
    got = binding.gated_scan_update(x, r, i, A, state, _ints([1, 1]), slots=_ints([entries - 1, -1]))
    assert torch.equal(want, got) and torch.equal(state[-1], near[0])


# ---- as many sequences as a wave has lanes, and more empty ones than that ----

@pytest.mark.parametrize("C", [1, 40])
@pytest.mark.parametrize("lens", [(3,) * 62, (1, 2, 0) * 21, (2, 1, 0, 1) * 16, (1,) * 65, (0,) * 100 + (3,) + (0,) * 150 + (70, 1) + (0,) * 90,
                                  (17,) + (0,) * 200 + (2, 0, 0, 30) * 20 + (0,) * 64], ids=lambda v: str(len(v)))
def test_counts_of_sequences(lens, C):
    log(f"[gated counts] {len(lens)} sequences C={C}")
    g = torch.Generator().manual_seed(len(lens))
    cu = R.sequences(lens, 2)
    T, n = cu[-1] + 3, len(lens)
    t = dict(x=_randn(g, T, C), r=_randn(g, T, C), i=_randn(g, T, C), A=-(0.05 + 3 * torch.rand(C, generator=g)))
    dout, state, dfin = _randn(g, T, C), _randn(g, n, C), _randn(g, n, C)
    seen = [k % 3 for k in range(n)]
    args = [t[k].cuda() for k in ("x", "r", "i", "A")]
    kept, dstate = torch.empty(-(-T // 64), C, device="cuda"), state.cuda()
    out = binding.gated_scan_varlen_fwd(*args, _ints(cu), state=dstate, cache_seqlens=_ints(seen), checkpoints=kept)
    ref, err, after, e_after = R.scan_cached(t, cu, state, seen, list(range(n)))
    R.close(out[2:-3], ref[2:-3], err[2:-3], f32, "out")
    R.close(dstate, after, e_after, f32, "cache")
    h0 = state * (torch.tensor(seen) > 0)[:, None]
    got = binding.gated_scan_varlen_bwd(*args, _ints(cu), dout.cuda(), kept, initial_states=h0.cuda(), dfinal_states=dfin.cuda(),
                                        want_dinitial_states=True)
    want = R.scan_bwd(t, cu, dout, h0, dfin)
    for k, v in got.items():
        R.close(v, *want[k], f32, k)
