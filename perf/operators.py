"""The operators of a Mamba-2 mixer's core, as they are measured: the short
causal convolution over packed tokens and its backward, the chunked scan of
packed prompts from and to a state cache, the same scan in training (the
chunks' states kept in 8 bits) with its backward, and the single-token step.

Plain forms in elementary torch operations, the framework's calls where
``own`` is set, and an exact value in 64 bits from the recurrence itself.
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

P = 64          # channels per head
Q = 64          # tokens per chunk; a checkpoint is the state entering a chunk
W = 4           # convolution taps
RING = 4        # entries of the convolution's ring cache
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # prompts of a chat batch entering the convolution of a small model, some of them continued
        dict(name="conv_chat", op="conv", tokens=3500, nseq=16, ragged=True, channels=2304, type="float16"),
        # the 2.7B-shaped layer's convolution over eight rows of 2048 tokens
        dict(name="conv_layer", op="conv", tokens=16384, nseq=8, ragged=False, channels=5376, type="bfloat16"),
        # its gradient in training
        dict(name="conv_bwd_layer", op="conv_bwd", tokens=16384, nseq=8, ragged=False, channels=5376, type="bfloat16"),
        # the gradient in a small fp32 experiment with an odd width
        dict(name="conv_bwd_odd", op="conv_bwd", tokens=2000, nseq=7, ragged=True, channels=1003, type="float32"),
        # prompts of a chat batch, gated, some continued from their cached state
        dict(name="scan_chat", op="scan", tokens=4100, nseq=24, ragged=True, heads=32, groups=1, dstate=128,
             gate=True, cache=True, train=False),
        # one long document through the 2.7B-shaped layer
        dict(name="scan_document", op="scan", tokens=32768, nseq=1, ragged=False, heads=80, groups=1, dstate=128,
             gate=False, cache=True, train=False),
        # the training forward of the 2.7B-shaped layer, keeping its 8-bit checkpoints
        dict(name="scan_train", op="scan", tokens=8192, nseq=4, ragged=False, heads=80, groups=1, dstate=128,
             gate=False, cache=False, train=True),
        # the training backward of the 2.7B-shaped layer
        dict(name="scan_bwd_layer", op="scan_bwd", tokens=16384, nseq=8, ragged=False, heads=80, groups=1, dstate=128),
        # the backward of a small grouped model on packed documents
        dict(name="scan_bwd_packed", op="scan_bwd", tokens=1000, nseq=5, ragged=True, heads=8, groups=2, dstate=64),
        # one user's next token in a small model: latency
        dict(name="step_one", op="step", batch=1, heads=32, groups=1, dstate=128, gate=False, type="bfloat16"),
        # a full serving batch through the 2.7B-shaped layer
        dict(name="step_batch", op="step", batch=128, heads=80, groups=1, dstate=128, gate=True, type="bfloat16"),
        # a middling batch of a grouped model, fp16
        dict(name="step_grouped", op="step", batch=33, heads=32, groups=4, dstate=64, gate=True, type="float16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "scan", "scan", "scan_bwd", "step"])
    if op in ("conv", "conv_bwd"):
        channels = rng.choice([_log_int(rng, 64, 5376), 8 * _log_int(rng, 8, 672)])
        tokens = _log_int(rng, 1, 16384)
        return dict(op=op, tokens=tokens, nseq=min(_log_int(rng, 1, 40), max(1, tokens // 2)), ragged=rng.random() < 0.7,
                    channels=channels, type=rng.choice(list(TYPES)))
    groups = rng.choice([1, 1, 2, 4])
    heads = groups * rng.choice([1, 2, 3, 5, 8, 10, 16, 20])
    dstate = rng.choice([32, 64, 128])
    if op == "step":
        return dict(op=op, batch=_log_int(rng, 1, 128), heads=heads, groups=groups, dstate=dstate,
                    gate=rng.random() < 0.5, type=rng.choice(list(TYPES)))
    tokens = _log_int(rng, 1, 16384)
    nseq = min(_log_int(rng, 1, 40), max(1, tokens // 2))
    case = dict(op=op, tokens=tokens, nseq=nseq, ragged=rng.random() < 0.7, heads=heads, groups=groups, dstate=dstate)
    if op == "scan":
        train = rng.random() < 0.4
        case.update(gate=rng.random() < 0.4, cache=not train, train=train)
    return case


def _lengths(case):
    """The sequences' lengths: equal, or ragged with an empty one and one of a
    single token among them where there are enough."""
    t, s = case["tokens"], case["nseq"]
    if not case["ragged"] or s == 1:
        return [t // s + (i < t % s) for i in range(s)]
    rng = random.Random(t * 8191 + s)
    cuts = sorted(rng.randint(0, t) for _ in range(s - 1))
    if s >= 5:
        cuts[0] = cuts[1]
        cuts[2] = min(cuts[1] + 1, cuts[3] if s > 4 else t)
        cuts.sort()
    return [b - a for a, b in zip([0] + cuts, cuts + [t])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sequences(case, st, gen, dev):
    lens = _lengths(case)
    s = len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["max_seqlen"] = max(lens)
    st["slots"] = torch.randperm(s + 2, generator=gen, device=dev)[:s].to(torch.int32)
    # every third request is a new one (nothing cached), the others continue
    seen = torch.randint(1, 5000, (s,), generator=gen, device=dev, dtype=torch.int32)
    st["seen"] = torch.where(torch.arange(s, device=dev) % 3 == 0, torch.zeros_like(seen), seen)


def _scan_params(case, st, gen, dev):
    h = case["heads"]
    st["A"] = -(1.0 + 15.0 * torch.rand(h, generator=gen, device=dev))
    st["D"] = torch.randn(h, generator=gen, device=dev)
    # steps log-uniform in [0.001, 0.1] at a zero projection, as these models are initialised
    step = torch.exp(torch.rand(h, generator=gen, device=dev) * math.log(100.0) + math.log(0.001))
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    st = {"op": op, "case": dict(case)}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if op in ("conv", "conv_bwd"):
        io, c, t = TYPES[case["type"]], case["channels"], case["tokens"]
        _sequences(case, st, gen, dev)
        st["x"] = normal(t, c).to(io)
        st["weight"], st["bias"] = 0.5 * normal(c, W), 0.1 * normal(c)
        if op == "conv":
            st["ring"] = normal(case["nseq"] + 2, c, RING).to(io)
        else:
            st["dout"] = normal(t, c).to(io)
        return st
    h, g, n = case["heads"], case["groups"], case["dstate"]
    _scan_params(case, st, gen, dev)
    if op == "step":
        io, b = TYPES[case["type"]], case["batch"]
        c = h * P + 2 * g * n
        # the input projection's row: gate | x B C | step
        row = normal(b, h * P + c + h).to(io)
        st["z"] = row[:, :h * P] if case["gate"] else None
        st["xbc"], st["dt"] = row[:, h * P:h * P + c], row[:, h * P + c:]
        st["weight"], st["bias"] = 0.5 * normal(c, W), 0.1 * normal(c)
        st["ring"] = normal(b + 2, c, RING).to(io)
        st["state"] = normal(b + 2, h, P, n)
        st["slots"] = torch.randperm(b + 2, generator=gen, device=dev)[:b].to(torch.int32)
        st["seen"] = torch.randint(1, 5000, (b,), generator=gen, device=dev, dtype=torch.int32)
        return st
    t = case["tokens"]
    _sequences(case, st, gen, dev)
    # x, B and C are parts of the convolution's output rows, as it leaves them
    xbc = F.silu(normal(t, h * P + 2 * g * n)).to(torch.bfloat16)
    st["x"] = xbc[:, :h * P].view(t, h, P)
    st["B"] = xbc[:, h * P:h * P + g * n].view(t, g, n)
    st["C"] = xbc[:, h * P + g * n:].view(t, g, n)
    st["dt"] = normal(t, h).to(torch.bfloat16)
    slots = t // Q + case["nseq"]
    if op == "scan":
        st["z"] = normal(t, h, P).to(torch.bfloat16) if case["gate"] else None
        st["state"] = normal(case["nseq"] + 2, h, P, n) if case["cache"] else None
        if case["train"]:
            st["codes"] = torch.zeros(slots, h, P, n, dtype=torch.int8, device=dev)
            st["scales"] = torch.ones(slots, h, P, device=dev)
        return st
    st["dout"] = normal(t, h, P).to(torch.bfloat16)
    states = _chunk_states(st, _slots(st["cu"], t))[0]
    st["codes"], st["scales"] = _to_8_bits(states)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _tokens(cu, t):
    """Each token's sequence and its place in it."""
    at = torch.arange(t, device=cu.device)
    seq = torch.searchsorted(cu.long(), at, right=True) - 1
    return at, seq, at - cu.long()[seq]


def _history(ring, slots, seen):
    """The three inputs before each sequence's first token, oldest first, zero
    before position 0: (nseq, 3, channels)."""
    pos = seen.long()[:, None] - 3 + torch.arange(3, device=ring.device)
    rows = ring[slots.long()].float().transpose(1, 2)
    got = torch.gather(rows, 1, (pos % RING)[..., None].expand(-1, -1, rows.shape[2]))
    return got * (pos >= 0)[..., None]


def _taps(x, cu, hist=None):
    """The four inputs that each token's output sees: (t, 4, channels)."""
    at, seq, pos = _tokens(cu, x.shape[0])
    k = torch.arange(W, device=x.device) - (W - 1)
    inside = (pos[:, None] + k >= 0)[..., None]
    v = x.float()[(at[:, None] + k).clamp(min=0)]
    if hist is None:
        return v * inside
    return torch.where(inside, v, hist[seq[:, None], (pos[:, None] + k + W - 1).clamp(max=W - 2)])


def _plain_conv(st):
    x, cu, ring = st["x"], st["cu"], st["ring"]
    v = _taps(x, cu, _history(ring, st["slots"], st["seen"]))
    out = F.silu((v * st["weight"].t()).sum(1) + st["bias"]).to(x.dtype)
    # the last tokens of each sequence into its ring
    lens = (cu[1:] - cu[:-1]).long()
    back = lens[:, None] - RING + torch.arange(RING, device=x.device)
    place = ((st["seen"].long()[:, None] + back) % RING)[:, None, :].expand(-1, x.shape[1], -1)
    rows = ring[st["slots"].long()]
    new = x[(cu[:-1].long()[:, None] + back).clamp(0, x.shape[0] - 1)].transpose(1, 2)
    kept = torch.where((back >= 0)[:, None, :], new, torch.gather(rows, 2, place))
    ring.index_copy_(0, st["slots"].long(), torch.scatter(rows, 2, place, kept))
    return {"out": out, "ring": ring}


def _plain_conv_bwd(st):
    x, cu, w = st["x"], st["cu"], st["weight"]
    t = x.shape[0]
    at, seq, pos = _tokens(cu, t)
    v = _taps(x, cu)
    pre = (v * w.t()).sum(1) + st["bias"]
    sig = torch.sigmoid(pre)
    da = st["dout"].float() * sig * (1.0 + pre * (1.0 - sig))
    ahead = torch.arange(W - 1, -1, -1, device=x.device)
    left = (cu.long()[1:][seq] - at)[:, None] > ahead
    later = da[(at[:, None] + ahead).clamp(max=t - 1)] * left[..., None]
    return {"dx": (later * w.t()).sum(1).to(x.dtype),
            "dweight": (da[:, None, :] * v).sum(0, dtype=torch.float64).t().float(),
            "dbias": da.sum(0, dtype=torch.float64).float()}


def _slots(cu, t):
    """The chunks of the packed sequences: chunk c of sequence s is slot
    cu[s] // Q + s + c.  Returns each slot's sequence, tokens and validity,
    each sequence's first slot, and each token's slot and place."""
    cu = cu.long()
    s = cu.shape[0] - 1
    base = cu[:-1] // Q + torch.arange(s, device=cu.device)
    slot = torch.arange(t // Q + s, device=cu.device)
    seq = torch.searchsorted(base, slot, right=True) - 1
    place = ((slot - base[seq]) * Q)[:, None] + torch.arange(Q, device=cu.device)
    valid = place < (cu[1:] - cu[:-1])[seq][:, None]
    tok = (cu[seq][:, None] + place).clamp(max=t - 1)
    _, tseq, pos = _tokens(cu, t)
    return {"seq": seq, "tok": tok, "valid": valid, "base": base, "tslot": base[tseq] + pos // Q, "tpos": pos % Q,
            "last": base + (cu[1:] - cu[:-1] - 1).clamp(min=0) // Q}


def _by_slot(v, sl):
    return v.float()[sl["tok"]] * sl["valid"].reshape(sl["valid"].shape + (1,) * (v.dim() - 1))


def _steps(st, sl):
    """dt', and the running sum of dt' A inside each chunk (64 bits)."""
    dt = F.softplus(_by_slot(st["dt"], sl) + st["dt_bias"]) * sl["valid"][..., None]
    return dt, torch.cumsum(dt.double() * st["A"].double(), 1)


def _between(cs, sl):
    """The decay from the end of each earlier slot to the start of a later one
    of the same sequence: (heads, slots, slots) and, from the sequence's
    start, (slots, heads)."""
    total = torch.cumsum(cs[:, -1], 0)
    before = total - cs[:, -1]
    same = sl["seq"][:, None] == sl["seq"][None, :]
    at = torch.arange(cs.shape[0], device=cs.device)
    earlier = same & (at[None, :] < at[:, None])
    d = torch.exp((before[:, None] - total[None, :]).masked_fill(~earlier[..., None], -math.inf)).float()
    return d.permute(2, 0, 1), torch.exp(before - before[sl["base"][sl["seq"]]]).float()


def _chunk_states(st, sl):
    """The state entering every chunk (slots, h, p, n), and each chunk's own
    end state from zero."""
    h = st["A"].shape[0]
    dt, cs = _steps(st, sl)
    x, b = _by_slot(st["x"], sl), _by_slot(st["B"], sl)
    weight = dt * torch.exp(cs[:, -1:] - cs).float()
    n = b.shape[-1]
    xw = (x * weight[..., None]).permute(0, 2, 3, 1)
    bh = b.repeat_interleave(h // b.shape[2], 2).permute(0, 2, 1, 3)
    ends = xw.contiguous() @ bh.contiguous()
    d, from_start = _between(cs, sl)
    states = (d.contiguous() @ ends.permute(1, 0, 2, 3).reshape(h, -1, P * n)).reshape(h, -1, P, n).permute(1, 0, 2, 3)
    if st.get("state") is not None:
        first = st["state"][st["slots"].long()] * (st["seen"] > 0)[:, None, None, None]
        states = states + from_start[..., None, None] * first[sl["seq"]]
    return states, ends


def _to_8_bits(states):
    top = states.abs().amax(-1)
    _, e = torch.frexp(top / 127.0)
    exact_power = top / 127.0 == torch.ldexp(torch.full_like(top, 0.5), e)
    scale = torch.ldexp(torch.ones_like(top), torch.where(exact_power, e - 1, e).clamp(-100, 127))
    return torch.round(states / scale[..., None]).to(torch.int8), scale


def _values(codes, scales):
    """What the 8-bit states stand for: a code times a power of two is exact
    in bfloat16."""
    return codes * scales.to(torch.bfloat16)[..., None]


def _lower(cs):
    """exp(cs_i - cs_j) for j <= i: (slots, heads, i, j)."""
    c = cs.permute(0, 2, 1)
    keep = torch.ones(Q, Q, dtype=torch.bool, device=cs.device).tril()
    return torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~keep, -math.inf)).float()


def _plain_scan(st):
    t, h, _ = st["x"].shape
    sl = _slots(st["cu"], t)
    dt, cs = _steps(st, sl)
    states, ends = _chunk_states(st, sl)
    x, b, c = (_by_slot(st[k], sl) for k in ("x", "B", "C"))
    rep = h // b.shape[2]
    s = c.permute(0, 2, 1, 3).contiguous() @ b.permute(0, 2, 3, 1).contiguous()
    m = s.repeat_interleave(rep, 1) * _lower(cs) * dt.permute(0, 2, 1)[:, :, None, :]
    y = m @ x.permute(0, 2, 1, 3).contiguous()
    ch = c.repeat_interleave(rep, 2).permute(0, 2, 1, 3)
    y = y + (ch.contiguous() @ states.transpose(2, 3).contiguous()) * torch.exp(cs).float().permute(0, 2, 1)[..., None]
    out = y[sl["tslot"], :, sl["tpos"]] + st["D"][:, None] * st["x"].float()
    if st["z"] is not None:
        out = out * F.silu(st["z"].float())
    r = {"out": out.to(torch.bfloat16)}
    if st["state"] is not None:
        total = torch.exp(cs[:, -1]).float()[..., None, None]
        st["state"].index_copy_(0, st["slots"].long(), (total * states + ends)[sl["last"]])
        r["state"] = st["state"]
    if "codes" in st:
        codes, scales = _to_8_bits(states)
        used = sl["valid"].any(1)   # slots past a sequence's last chunk keep what they hold
        r["checkpoints"] = _values(torch.where(used[:, None, None, None], codes, st["codes"]),
                                   torch.where(used[:, None, None], scales, st["scales"]))
    return r


def _plain_scan_bwd(st):
    t, h, _ = st["x"].shape
    sl = _slots(st["cu"], t)
    dt, cs = _steps(st, sl)
    x, b, c, g = (_by_slot(st[k], sl) for k in ("x", "B", "C", "dout"))
    groups, n = b.shape[2], b.shape[3]
    rep = h // groups
    heads = lambda v: v.permute(0, 2, 1, 3).contiguous()  # noqa: E731
    x, g, bh, ch = heads(x), heads(g), heads(b.repeat_interleave(rep, 2)), heads(c.repeat_interleave(rep, 2))
    hs = st["codes"].float() * st["scales"][..., None]
    e, w, total = (torch.exp(v).float().permute(0, 2, 1) for v in (cs, cs[:, -1:] - cs, cs[:, -1:]))
    dts = dt.permute(0, 2, 1)
    # the adjoint of the state leaving every chunk
    own_part = (g * e[..., None]).transpose(2, 3).contiguous() @ ch
    d, _ = _between(cs, sl)
    dh = (d.transpose(1, 2).contiguous() @ own_part.permute(1, 0, 2, 3).reshape(h, -1, P * n)).reshape(h, -1, P, n)
    dh = dh.permute(1, 0, 2, 3).contiguous()
    low = _lower(cs)
    s = (heads(c) @ heads(b).transpose(2, 3).contiguous()).repeat_interleave(rep, 1)
    m = (g @ x.transpose(2, 3).contiguous()) * low
    pair = s * m
    db_state = (x @ dh) * w[..., None]
    dc_state = (g @ hs) * e[..., None]
    dx = (s * low).transpose(2, 3).contiguous() @ g + (bh @ dh.transpose(2, 3).contiguous()) * w[..., None]
    dx = dx * dts[..., None] + st["D"][:, None, None] * g
    mv = m * dts[:, :, None, :]
    dc = mv @ bh + dc_state
    db = mv.transpose(2, 3).contiguous() @ ch + db_state * dts[..., None]
    # the steps: through the inputs' weights, and through every decay
    direct = pair.sum(2) + (db_state * bh).sum(-1)
    dcs = ((pair * dts[:, :, None, :]).sum(3) + (dc_state * ch).sum(-1)).double() - (dts * direct).double()
    through = (dts * (db_state * bh).sum(-1)).double().sum(-1) + total[..., 0] * (dh * hs).double().sum((2, 3))
    dcs[..., -1] += through
    da = torch.flip(torch.cumsum(torch.flip(dcs, (2,)), 2), (2,))
    ddt = direct + st["A"][:, None] * da.float()
    sig = torch.sigmoid(_by_slot(st["dt"], sl) + st["dt_bias"]).permute(0, 2, 1) * sl["valid"][:, None]
    ddt = ddt * sig
    back = lambda v: v[sl["tslot"], :, sl["tpos"]]  # noqa: E731
    per_group = lambda v: v.reshape(v.shape[0], groups, rep, Q, n).sum(2)  # noqa: E731
    bf = torch.bfloat16
    return {"dx": back(dx).to(bf), "ddt": back(ddt).to(bf), "dB": back(per_group(db)).to(bf),
            "dC": back(per_group(dc)).to(bf), "dA": (dts.double() * da).sum((0, 2)).float(),
            "dD": (g * x).sum(-1).double().sum((0, 2)).float(), "ddt_bias": ddt.double().sum((0, 2)).float()}


def _plain_step(st):
    xbc, ring, state, h = st["xbc"], st["ring"], st["state"], st["A"].shape[0]
    n, slots, seen = state.shape[3], st["slots"].long(), st["seen"].long()
    g = (xbc.shape[1] - h * P) // (2 * n)
    hist = _history(ring, st["slots"], st["seen"])
    v = torch.cat([hist, xbc.float()[:, None]], 1)
    u = F.silu((v * st["weight"].t()).sum(1) + st["bias"])
    ring[slots, :, seen % RING] = xbc
    x = u[:, :h * P].reshape(-1, h, P)
    b, c = (u[:, h * P + k * g * n:h * P + (k + 1) * g * n].reshape(-1, g, n).repeat_interleave(h // g, 1) for k in (0, 1))
    dt = F.softplus(st["dt"].float() + st["dt_bias"])
    old = state[slots] * (seen > 0)[:, None, None, None]
    new = torch.exp(dt * st["A"])[..., None, None] * old + (dt[..., None] * x)[..., None] * b[:, :, None, :]
    state.index_copy_(0, slots, new)
    y = (new * c[:, :, None, :]).sum(-1) + st["D"][:, None] * x
    y = y.reshape(-1, h * P)
    if st["z"] is not None:
        y = y * F.silu(st["z"].float())
    return {"out": y.to(xbc.dtype), "state": state, "ring": ring}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(st):
    from state_space_model_scan_amd import binding as ssm
    op = st["op"]
    if op == "conv":
        out = ssm.causal_conv1d_varlen_fwd(st["x"], st["weight"], st["cu"], bias=st["bias"], activation="silu",
                                           conv_state=st["ring"], cache_seqlens=st["seen"], slots=st["slots"])
        return {"out": out, "ring": st["ring"]}
    if op == "conv_bwd":
        return ssm.causal_conv1d_varlen_bwd(st["x"], st["weight"], st["cu"], st["dout"], bias=st["bias"],
                                            activation="silu")
    if op == "step":
        out = ssm.conv1d_ssd_update(st["xbc"], st["dt"], st["A"], st["weight"], st["ring"], st["state"], st["seen"],
                                    conv_bias=st["bias"], D=st["D"], z=st["z"], dt_bias=st["dt_bias"], dt_softplus=True,
                                    slots=st["slots"])
        return {"out": out, "state": st["state"], "ring": st["ring"]}
    if op == "scan":
        r = {}
        kw = {}
        if st["state"] is not None:
            kw.update(ssm_state=st["state"], cache_seqlens=st["seen"], slots=st["slots"])
        if "codes" in st:
            kw.update(checkpoints=(st["codes"], st["scales"]))
        r["out"] = ssm.ssd_varlen_fwd(st["x"], st["dt"], st["A"], st["B"], st["C"], st["cu"], st["max_seqlen"], D=st["D"],
                                      z=st["z"], dt_bias=st["dt_bias"], dt_softplus=True, **kw)
        if st["state"] is not None:
            r["state"] = st["state"]
        if "codes" in st:
            r["checkpoints"] = _values(st["codes"], st["scales"])
        return r
    return ssm.ssd_varlen_bwd(st["x"], st["dt"], st["A"], st["B"], st["C"], st["cu"], st["max_seqlen"], st["dout"],
                              (st["codes"], st["scales"]), D=st["D"], dt_bias=st["dt_bias"], dt_softplus=True)


def run(st):
    if own:
        return _own(st)
    return {"conv": _plain_conv, "conv_bwd": _plain_conv_bwd, "scan": _plain_scan, "scan_bwd": _plain_scan_bwd,
            "step": _plain_step}[st["op"]](st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("conv", "conv_bwd"):
        size = 4 if case["type"] == "float32" else 2
        io = case["tokens"] * case["channels"]
        par = case["channels"] * (W + 1) * 4
        if op == "conv":
            return {"bytes": 2 * size * io + par + 2 * case["nseq"] * case["channels"] * RING * size, "flops": 14 * io}
        return {"bytes": 3 * size * io + 2 * par, "flops": 36 * io}
    h, g, n = case["heads"], case["groups"], case["dstate"]
    if op == "step":
        size = 4 if case["type"] == "float32" else 2
        b, c = case["batch"], h * P + 2 * g * n
        row = c * (1 + RING + 1) + h + h * P * (2 if case["gate"] else 1)
        return {"bytes": b * (2 * h * P * n * 4 + row * size) + c * (W + 1) * 4 + 3 * h * 4, "flops": b * h * P * n * 6}
    t = case["tokens"]
    chunks = sum(-(-v // Q) for v in _lengths(case))
    row, bc = h * P * 2, g * n * 2
    held = chunks * h * P * (n + 4)
    # multiply-adds of one chunk and head: the lower half of the token pairs, and the products with a state
    pairs, wide = Q * Q / 2, Q * P * n
    if op == "scan":
        state = 2 * case["nseq"] * h * P * n * 4 if case["cache"] else 0
        return {"bytes": t * (row * (3 if case["gate"] else 2) + 2 * bc + 2 * h) + state + (held if case["train"] else 0),
                "flops": 2 * chunks * (h * (pairs * P + 2 * wide) + g * pairs * n)}
    return {"bytes": t * (3 * row + 4 * bc + 4 * h) + held,
            "flops": 2 * chunks * (h * (2 * pairs * P + 4 * wide) + 3 * g * pairs * n)}


# ---------------------------------------------------------------------------
# exact values: the recurrences themselves, token by token, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op in ("scan", "scan_bwd"):
        longest = max(_lengths(case))
        bytes_a_step = case["nseq"] * case["heads"] * P * case["dstate"] * 8
        if longest * (bytes_a_step * (60 if op == "scan_bwd" else 16) / 3e12 + (80 if op == "scan_bwd" else 20) * 1e-5) > 15:
            return None
    st = prepare(case, seed)
    return {"conv": _exact_conv, "conv_bwd": _exact_conv_bwd, "scan": _exact_scan, "scan_bwd": _exact_scan_bwd,
            "step": _exact_step}[op](st)


def _cut(cu):
    edges = cu.tolist()
    return list(zip(edges[:-1], edges[1:]))


def _padded(x, before):
    """x of one sequence in 64 bits with the three inputs before it."""
    return torch.cat([before.to(torch.float64), x.to(torch.float64)])


def _before(st, s):
    c, dev = st["x"].shape[1], st["x"].device
    rows = torch.zeros(W - 1, c, dtype=torch.float64, device=dev)
    if "ring" in st:
        seen, slot = int(st["seen"][s]), int(st["slots"][s])
        for j in range(W - 1):
            if seen - (W - 1) + j >= 0:
                rows[j] = st["ring"][slot, :, (seen - (W - 1) + j) % RING].double()
    return rows


def _conv64(v, weight, bias):
    n = v.shape[0] - (W - 1)
    return sum(v[k:k + n] * weight[:, k].double() for k in range(W)) + bias.double()


def _exact_conv(st):
    x, outs, ring = st["x"], [], st["ring"].double()
    for s, (a, b) in enumerate(_cut(st["cu"])):
        pre = _conv64(_padded(x[a:b], _before(st, s)), st["weight"], st["bias"])
        outs.append(pre / (1.0 + torch.exp(-pre)))
    for s, (a, b) in enumerate(_cut(st["cu"])):
        for i in range(max(a, b - RING), b):
            ring[int(st["slots"][s]), :, (int(st["seen"][s]) + i - a) % RING] = x[i].double()
    return {"out": torch.cat(outs), "ring": ring}


def _exact_conv_bwd(st):
    w = st["weight"].double()
    dx, dw, db = [], torch.zeros_like(w), torch.zeros_like(st["bias"].double())
    for s, (a, b) in enumerate(_cut(st["cu"])):
        v = _padded(st["x"][a:b], _before(st, s))
        pre = _conv64(v, st["weight"], st["bias"])
        sig = 1.0 / (1.0 + torch.exp(-pre))
        da = st["dout"][a:b].double() * (sig + pre * sig * (1.0 - sig))
        part = torch.zeros_like(v)
        for k in range(W):
            part[k:k + b - a] += da * w[:, k]
            dw[:, k] += (da * v[k:k + b - a]).sum(0)
        dx.append(part[W - 1:])
        db += da.sum(0)
    return {"dx": torch.cat(dx), "dweight": dw, "dbias": db}


def _rows64(st, v):
    """Packed tokens as rows, one for each sequence, zero behind its end."""
    cuts = _cut(st["cu"])
    out = torch.zeros((len(cuts), max(st["max_seqlen"], 1)) + tuple(v.shape[1:]), dtype=torch.float64, device=v.device)
    for s, (a, b) in enumerate(cuts):
        out[s, :b - a] = v[a:b].double()
    return out


def _packed64(st, rows):
    return torch.cat([rows[s, :b - a] for s, (a, b) in enumerate(_cut(st["cu"]))])


def _softplus64(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)


def _live(st):
    cu = st["cu"].long()
    return torch.arange(max(st["max_seqlen"], 1), device=cu.device)[None, :] < (cu[1:] - cu[:-1])[:, None]


def _exact_scan(st):
    h, live = st["A"].shape[0], _live(st)
    x, b, c = (_rows64(st, st[k]) for k in ("x", "B", "C"))
    rep = h // b.shape[2]
    dt = _softplus64(_rows64(st, st["dt"]) + st["dt_bias"].double()) * live[..., None]
    keep = torch.exp(dt * st["A"].double())
    s, n = x.shape[0], b.shape[3]
    state = torch.zeros(s, h, P, n, dtype=torch.float64, device=x.device)
    if st["state"] is not None:
        for i in range(s):
            if int(st["seen"][i]) > 0:
                state[i] = st["state"][int(st["slots"][i])].double()
    y = torch.zeros_like(x)
    held = {}
    for t in range(x.shape[1]):
        if "codes" in st and t % Q == 0:
            held[t // Q] = state.float()
        bt = b[:, t].repeat_interleave(rep, 1)
        state.mul_(keep[:, t, :, None, None]).addcmul_((dt[:, t, :, None] * x[:, t])[..., None], bt[:, :, None, :])
        y[:, t] = torch.matmul(state, c[:, t].repeat_interleave(rep, 1)[..., None])[..., 0]
    out = _packed64(st, y + st["D"].double()[:, None] * x)
    if st["z"] is not None:
        z = st["z"].double()
        out = out * z / (1.0 + torch.exp(-z))
    r = {"out": out}
    if st["state"] is not None:
        end = st["state"].double()
        for i in range(s):
            end[int(st["slots"][i])] = state[i]
        r["state"] = end
    if "codes" in st:
        # the steps of a code are far wider than 32 bits' rounding; only ties near a border can fall the other way
        values = torch.zeros(st["codes"].shape, dtype=torch.float64, device=x.device)
        for i, (a, e) in enumerate(_cut(st["cu"])):
            for k in range(-(-(e - a) // Q)):
                v = held[k][i].double()
                top = v.abs().amax(-1, keepdim=True)
                scale = torch.exp2(torch.ceil(torch.log2((top / 127.0).clamp(min=2.0 ** -100))))
                values[a // Q + i + k] = torch.round(v / scale) * scale
        r["checkpoints"] = values
    return r


def _exact_scan_bwd(st):
    h, live = st["A"].shape[0], _live(st)
    x, b, c, g = (_rows64(st, st[k]) for k in ("x", "B", "C", "dout"))
    raw = _rows64(st, st["dt"]) + st["dt_bias"].double()
    dt = _softplus64(raw) * live[..., None]
    a_log = st["A"].double()
    keep = torch.exp(dt * a_log)
    s, length, groups, n = x.shape[0], x.shape[1], b.shape[2], b.shape[3]
    rep = h // groups
    adj = torch.zeros(s, h, P, n, dtype=torch.float64, device=x.device)
    dx, ddt, db, dc = torch.zeros_like(x), torch.zeros_like(dt), torch.zeros_like(b), torch.zeros_like(c)
    d_a = torch.zeros_like(a_log)
    cuts = _cut(st["cu"])
    for k in range((length - 1) // Q, -1, -1):
        state = torch.zeros_like(adj)
        for i, (lo, hi) in enumerate(cuts):
            if k * Q < hi - lo:
                at = lo // Q + i + k
                state[i] = st["codes"][at].double() * st["scales"][at].double()[..., None]
        steps = range(k * Q, min(length, (k + 1) * Q))
        states = []
        for t in steps:
            states.append(state)
            bt = b[:, t].repeat_interleave(rep, 1)
            state = state * keep[:, t, :, None, None]
            state.addcmul_((dt[:, t, :, None] * x[:, t])[..., None], bt[:, :, None, :])
        for t in reversed(steps):
            bt, ct = b[:, t].repeat_interleave(rep, 1), c[:, t].repeat_interleave(rep, 1)
            gt, xt, dtt = g[:, t], x[:, t], dt[:, t]
            dc[:, t] = torch.matmul(gt[:, :, None, :], state)[:, :, 0].reshape(s, groups, rep, n).sum(2)
            adj.addcmul_(gt[..., None], ct[:, :, None, :])
            adj_b = torch.matmul(adj, bt[..., None])[..., 0]
            state = states[t - k * Q]
            dx[:, t] = dtt[..., None] * adj_b
            db[:, t] = (dtt[..., None] * torch.matmul(xt[:, :, None, :], adj)[:, :, 0]).reshape(s, groups, rep, n).sum(2)
            decayed = keep[:, t] * (adj * state).sum((2, 3))
            ddt[:, t] = (adj_b * xt).sum(-1) + a_log * decayed
            d_a += (dtt * decayed).sum(0)
            adj.mul_(keep[:, t, :, None, None])
    dx = dx + st["D"].double()[:, None] * g
    ddt = ddt / (1.0 + torch.exp(-raw)) * live[..., None]
    return {"dx": _packed64(st, dx), "ddt": _packed64(st, ddt), "dB": _packed64(st, db), "dC": _packed64(st, dc),
            "dA": d_a, "dD": (g * x).sum((0, 1, 3)), "ddt_bias": ddt.sum((0, 1))}


def _exact_step(st):
    ring, state = st["ring"].double(), st["state"].double()
    h, n = st["A"].shape[0], state.shape[3]
    xbc = st["xbc"].double()
    g = (xbc.shape[1] - h * P) // (2 * n)
    outs = []
    for i, (slot, seen) in enumerate(zip(st["slots"].tolist(), st["seen"].tolist())):
        ring[slot, :, seen % RING] = xbc[i]
        u = st["bias"].double().clone()
        for k in range(W):
            if seen - (W - 1) + k >= 0:
                u += st["weight"][:, k].double() * ring[slot, :, (seen - (W - 1) + k) % RING]
        u = u / (1.0 + torch.exp(-u))
        x, b, c = u[:h * P].reshape(h, P), u[h * P:h * P + g * n].reshape(g, n), u[h * P + g * n:].reshape(g, n)
        b, c = b.repeat_interleave(h // g, 0), c.repeat_interleave(h // g, 0)
        dt = _softplus64(st["dt"][i].double() + st["dt_bias"].double())
        if seen == 0:
            state[slot] = 0.0
        state[slot] *= torch.exp(dt * st["A"].double())[:, None, None]
        state[slot] += (dt[:, None] * x)[:, :, None] * b[:, None, :]
        y = (state[slot] * c[:, None, :]).sum(-1) + st["D"].double()[:, None] * x
        y = y.reshape(-1)
        if st["z"] is not None:
            z = st["z"][i].double()
            y = y * z / (1.0 + torch.exp(-z))
        outs.append(y)
    return {"out": torch.stack(outs), "state": state, "ring": ring}
