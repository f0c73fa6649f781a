"""The operators of a gated recurrent block, as they are measured: the gated
linear recurrence over packed tokens from and to a state cache, the same in
training with its backward, its single-token step, and the block's
root-mean-square norm (with the residual's addition or a gate before it, to the
activations' type or to 8 bits with scales) with its backward.

Plain forms in elementary torch operations, the framework's calls where
``own`` is set, and an exact value in 64 bits from the definitions.

The recurrence, for every channel, with sigma the logistic function:
    rho = sigma(r + r_bias), iota = sigma(i + i_bias), a = exp(A rho)
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) iota_t x_t
The norm, over a group of n neighbouring columns:
    v = x, x + residual, or x silu(z);  y = v / sqrt(mean v^2 + eps) weight
"""
import math
import random

import torch

own = False

CHUNK = 64      # tokens from one kept state of the recurrence to the next
BLOCK = 128     # columns that share a scale in 8 bits
E4M3_MAX = 448.0
EPS = 1e-5
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # prompts of a chat batch through a small model's recurrence, some of them continued
        dict(name="scan_chat", op="scan", tokens=4100, nseq=24, ragged=True, channels=2304, type="float16", cache=True,
             train=False),
        # the training forward over eight rows of 2048 tokens, keeping the states that its backward starts from
        dict(name="scan_layer", op="scan", tokens=16384, nseq=8, ragged=False, channels=2560, type="bfloat16", cache=False,
             train=True),
        # one long document
        dict(name="scan_document", op="scan", tokens=65536, nseq=1, ragged=False, channels=2560, type="bfloat16", cache=True,
             train=False),
        # the training backward of the layer
        dict(name="scan_bwd_layer", op="scan_bwd", tokens=16384, nseq=8, ragged=False, channels=2560, type="bfloat16"),
        # the backward of a small fp32 experiment on packed documents, with an odd width
        dict(name="scan_bwd_odd", op="scan_bwd", tokens=2000, nseq=7, ragged=True, channels=1003, type="float32"),
        # one user's next token: latency
        dict(name="step_one", op="step", batch=1, channels=2560, type="bfloat16"),
        # a full serving batch of a wide layer
        dict(name="step_batch", op="step", batch=256, channels=5120, type="bfloat16"),
        # a few requests' tokens entering a block: the residual stream and the norm, latency
        dict(name="norm_tokens", op="norm", rows=16, cols=2560, groups=1, type="bfloat16", residual="bfloat16", gate=False,
             quant=False),
        # prompts of a chat batch entering a block whose products take 8 bits
        dict(name="norm_prompts", op="norm", rows=4100, cols=2560, groups=1, type="bfloat16", residual="bfloat16",
             gate=False, quant=True),
        # the gated norm of a wide mixer in training, eight groups of a row
        dict(name="norm_gated", op="norm", rows=16384, cols=5120, groups=8, type="bfloat16", residual="", gate=True,
             quant=False),
        # the training backward of a block's norm, the residual stream in 32 bits
        dict(name="norm_bwd_layer", op="norm_bwd", rows=16384, cols=2560, groups=1, type="bfloat16", residual="float32",
             gate=False),
        # the backward of a gated norm in a small fp32 experiment, odd groups
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1500, cols=1001, groups=7, type="float32", residual="", gate=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_bwd", "step", "norm", "norm", "norm_bwd"])
    wide = rng.choice([_log_int(rng, 64, 5120), 8 * _log_int(rng, 8, 640)])
    io = rng.choice(list(TYPES))
    if op == "step":
        return dict(op=op, batch=_log_int(rng, 1, 256), channels=wide, type=io)
    if op in ("scan", "scan_bwd"):
        tokens = _log_int(rng, 1, 16384)
        case = dict(op=op, tokens=tokens, nseq=min(_log_int(rng, 1, 40), max(1, tokens // 2)), ragged=rng.random() < 0.7,
                    channels=wide, type=io)
        if op == "scan":
            train = rng.random() < 0.4
            case.update(cache=not train, train=train)
        return case
    gate = rng.random() < 0.4
    groups = rng.choice([1, 2, 4, 8]) if gate else 1
    quant = op == "norm" and rng.random() < 0.4
    per = max(8, wide // groups)
    if quant and groups > 1:
        per = BLOCK * max(1, per // BLOCK)
    case = dict(op=op, rows=_log_int(rng, 1, 16384), cols=per * groups, groups=groups, type=io,
                residual="" if gate else rng.choice(["", io, io, "float32"]), gate=gate)
    if op == "norm":
        case["quant"] = quant
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
        cuts[2] = min(cuts[1] + 1, cuts[3])
    return [b - a for a, b in zip([0] + cuts, cuts + [t])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    op, io = case["op"], TYPES[case["type"]]
    st = {"op": op}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if op in ("norm", "norm_bwd"):
        t, c = case["rows"], case["cols"]
        res = TYPES.get(case["residual"])
        st["group"] = c // case["groups"]
        st["weight"] = 1.0 + 0.2 * normal(c)
        # a residual stream grows with the layers that have added to it
        st["x"] = normal(t, c).to(io)
        st["residual"] = (4.0 * normal(t, c)).to(res) if res else None
        # the gate is a part of the input projection's row, as it leaves it
        st["z"] = normal(t, c + 64).to(io)[:, :c] if case["gate"] else None
        if op == "norm":
            st["quant"] = case["quant"]
            return st
        if res:   # what the forward left, and the gradient that comes along the residual stream
            st["x"] = (st["x"].float() + st.pop("residual").float()).to(res)
            st["ds"] = normal(t, c).to(res)
        else:
            st["ds"] = None
        st["dy"] = normal(t, c).to(io)
        return st

    c = case["channels"]
    # exp(A / 8) is uniform in [0.9, 0.999], as these layers are initialised
    st["A"] = 8.0 * torch.log(0.9 + 0.099 * torch.rand(c, generator=gen, device=dev))
    st["r_bias"], st["i_bias"] = 0.5 * normal(c), 0.5 * normal(c)
    if op == "step":
        b = case["batch"]
        # the two gates lie side by side, as their projection leaves them
        gates = normal(b, 2 * c).to(io)
        st["x"], st["r"], st["i"] = normal(b, c).to(io), gates[:, :c], gates[:, c:]
        st["state"] = normal(b + 2, c)
        st["slots"] = torch.randperm(b + 2, generator=gen, device=dev)[:b].to(torch.int32)
        st["seen"] = torch.randint(1, 5000, (b,), generator=gen, device=dev, dtype=torch.int32)
        return st
    t = case["tokens"]
    lens = _lengths(case)
    s = len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st["cu"], st["longest"] = torch.tensor(cu, dtype=torch.int32, device=dev), max(lens)
    gates = normal(t, 2 * c).to(io)
    st["x"], st["r"], st["i"] = normal(t, c).to(io), gates[:, :c], gates[:, c:]
    if op == "scan_bwd":
        st["dout"] = normal(t, c).to(io)
        st["held"] = _held(_states(st, _gates(st))[1])
        return st
    st["held"] = torch.zeros(-(-t // CHUNK), c, device=dev) if case["train"] else None
    st["state"] = None
    if case["cache"]:
        st["state"] = normal(s + 2, c)
        st["slots"] = torch.randperm(s + 2, generator=gen, device=dev)[:s].to(torch.int32)
        # every third request is a new one (nothing cached), the others continue
        seen = torch.randint(1, 5000, (s,), generator=gen, device=dev, dtype=torch.int32)
        st["seen"] = torch.where(torch.arange(s, device=dev) % 3 == 0, torch.zeros_like(seen), seen)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _gates(st):
    """rho, iota, a and the weight sqrt(1 - a^2) of every token and channel."""
    rho, iota = _sigmoid(st["r"].float() + st["r_bias"]), _sigmoid(st["i"].float() + st["i_bias"])
    log_a = st["A"] * rho
    return rho, iota, torch.exp(log_a), torch.sqrt(-torch.expm1(2.0 * log_a))


def _running(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the tokens, spans doubled step by step; a
    factor of 0 starts a sequence."""
    span = 1
    while span < longest:
        b = torch.cat([b[:span], torch.addcmul(b[span:], a[span:], b[:-span])])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _edges(cu, t):
    """Each token's sequence, and whether it is the first and the last of it."""
    at, cu = torch.arange(t, device=cu.device), cu.long()
    seq = torch.searchsorted(cu, at, right=True) - 1
    return seq, at == cu[seq], at + 1 == cu[seq + 1]


def _states(st, gates):
    """The state after every token and the one before it."""
    _, iota, a, m = gates
    seq, first, _ = _edges(st["cu"], a.shape[0])
    start = torch.zeros((), device=a.device)
    if st.get("state") is not None:
        start = (st["state"][st["slots"].long()] * (st["seen"] > 0)[:, None])[seq]
    first = first[:, None]
    b = m * (iota * st["x"].float())
    h = _running(torch.where(first, 0.0, a), torch.where(first, torch.addcmul(b, a, start), b), st["longest"])
    before = torch.where(first, start, torch.cat([h[:1], h[:-1]]))
    return h, before


def _held(before):
    return before[::CHUNK].contiguous()


def _plain_scan(st):
    h, before = _states(st, _gates(st))
    r = {"out": h.to(st["x"].dtype)}
    if st["state"] is not None:
        seq, _, last = _edges(st["cu"], h.shape[0])
        length = (st["cu"][1:] - st["cu"][:-1]).long()
        ends = h[(st["cu"][1:].long() - 1).clamp(min=0)]
        slots = st["slots"].long()
        st["state"].index_copy_(0, slots, torch.where((length > 0)[:, None], ends, st["state"][slots]))
        r["state"] = st["state"]
    if st["held"] is not None:
        r["held"] = _held(before)
    return r


def _plain_scan_bwd(st):
    rho, iota, a, m = gates = _gates(st)
    x, g = st["x"].float(), st["dout"].float()
    before = _states(st, gates)[1]
    # the adjoint, against the tokens' order: G_t = dout_t + a_{t+1} G_{t+1}
    last = _edges(st["cu"], x.shape[0])[2][:, None]
    after = torch.where(last, 0.0, torch.cat([a[1:], a[:1]]))
    adj = torch.flip(_running(torch.flip(after, (0,)), torch.flip(g, (0,)), st["longest"]), (0,))
    gated = iota * x
    # rho dL/d(log a): through the state's factor and through the input's weight
    q = adj * rho * (a * before - a * a * gated / m)
    dr = st["A"] * (1.0 - rho) * q
    dx = adj * m * iota
    di = adj * m * gated * (1.0 - iota)
    io = st["x"].dtype
    total = lambda v: v.sum(0, dtype=torch.float64).float()  # noqa: E731
    return {"dx": dx.to(io), "dr": dr.to(io), "di": di.to(io), "dA": total(q), "dr_bias": total(dr), "di_bias": total(di)}


def _plain_step(st):
    _, iota, a, m = _gates(st)
    slots = st["slots"].long()
    h = torch.addcmul(m * (iota * st["x"].float()), a, st["state"][slots] * (st["seen"] > 0)[:, None])
    st["state"].index_copy_(0, slots, h)
    return {"out": h.to(st["x"].dtype), "state": st["state"]}


def _values(codes, scales):
    """What the 8-bit outputs stand for: a code times a power of two, exact in
    bfloat16."""
    rows, cols = codes.shape
    if cols % BLOCK == 0:
        return (codes.to(torch.bfloat16).view(rows, -1, BLOCK) * scales.to(torch.bfloat16)[..., None]).view(rows, cols)
    return codes.to(torch.bfloat16) * scales.to(torch.bfloat16).repeat_interleave(BLOCK, 1)[:, :cols]


def _to_8_bits(y):
    """Codes and scales of y: for every 128 columns of a row the smallest power
    of two (at least 2^-100) with which none of them is over 448."""
    rows, cols = y.shape
    pad = -cols % BLOCK
    wide = torch.cat([y, y.new_zeros(rows, pad)], 1).view(rows, -1, BLOCK)
    frac, e = torch.frexp(wide.abs().amax(-1) / E4M3_MAX)
    scale = torch.ldexp(torch.ones_like(frac), torch.where(frac == 0.5, e - 1, e).clamp(min=-100))
    return (wide / scale[..., None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn), scale


def _plain_norm(st):
    x, w, n = st["x"], st["weight"], st["group"]
    r = {}
    v = x.float()
    if st["residual"] is not None:
        r["residual"] = (v + st["residual"].float()).to(st["residual"].dtype)
        v = r["residual"].float()
    if st["z"] is not None:
        z = st["z"].float()
        v = v * (z * _sigmoid(z))
    by = v.view(v.shape[0], -1, n)
    y = (by / torch.sqrt((by * by).mean(-1, keepdim=True) + EPS)).view_as(v) * w
    if st["quant"]:
        r["out"] = _values(*_to_8_bits(y))
    else:
        r["out"] = y.to(x.dtype)
    return r


def _plain_norm_bwd(st):
    x, n, io = st["x"].float(), st["group"], st["dy"].dtype
    gate = 1.0
    if st["z"] is not None:
        z = st["z"].float()
        sig = _sigmoid(z)
        gate = z * sig
    by = (x * gate).view(x.shape[0], -1, n)
    rstd = 1.0 / torch.sqrt((by * by).mean(-1, keepdim=True) + EPS)
    hat = by * rstd
    dy = st["dy"].float()
    g = (dy * st["weight"]).view_as(by)
    dv = (rstd * (g - hat * (g * hat).mean(-1, keepdim=True))).view_as(x)
    r = {"dweight": (dy * hat.view_as(x)).sum(0, dtype=torch.float64).float()}
    if st["z"] is not None:
        r["dz"] = (dv * x * (sig * (1.0 + z * (1.0 - sig)))).to(io)
    dx = dv * gate
    if st["ds"] is not None:
        dx = dx + st["ds"].float()
        if st["ds"].dtype != io:
            r["dresidual"] = dx.to(st["ds"].dtype)
    r["dx"] = dx.to(io)
    return r


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(st):
    from state_space_model_scan_amd import binding as ssm
    op = st["op"]
    if op == "norm":
        kw = dict(residual=st["residual"], z=st["z"], group_size=st["group"], eps=EPS)
        if st["quant"]:
            codes, scales, *kept = ssm.rms_norm_quant_fwd(st["x"], st["weight"], **kw)
            r = {"out": _values(codes, scales)}
        else:
            got = ssm.rms_norm_fwd(st["x"], st["weight"], **kw)
            out, *kept = (got,) if st["residual"] is None else got
            r = {"out": out}
        if st["residual"] is not None:
            r["residual"] = kept[0]
        return r
    if op == "norm_bwd":
        return ssm.rms_norm_bwd(st["x"], st["weight"], st["dy"], z=st["z"], ds=st["ds"], group_size=st["group"], eps=EPS)
    gates = dict(r_bias=st["r_bias"], i_bias=st["i_bias"])
    if op == "step":
        out = ssm.gated_scan_update(st["x"], st["r"], st["i"], st["A"], st["state"], st["seen"], slots=st["slots"], **gates)
        return {"out": out, "state": st["state"]}
    if op == "scan":
        if st["state"] is not None:
            gates.update(state=st["state"], cache_seqlens=st["seen"], slots=st["slots"])
        r = {"out": ssm.gated_scan_varlen_fwd(st["x"], st["r"], st["i"], st["A"], st["cu"], checkpoints=st["held"], **gates)}
        if st["state"] is not None:
            r["state"] = st["state"]
        if st["held"] is not None:
            r["held"] = st["held"]
        return r
    return ssm.gated_scan_varlen_bwd(st["x"], st["r"], st["i"], st["A"], st["cu"], st["dout"], st["held"], **gates)


def run(st):
    if own:
        return _own(st)
    return {"scan": _plain_scan, "scan_bwd": _plain_scan_bwd, "step": _plain_step, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd}[st["op"]](st)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, size = case["op"], 4 if case["type"] == "float32" else 2
    if op in ("norm", "norm_bwd"):
        n, c = case["rows"] * case["cols"], case["cols"]
        stream = {"": 0, "float32": 4, "bfloat16": 2, "float16": 2}[case["residual"]]
        if op == "norm":
            scales = case["rows"] * -(-c // BLOCK) * 4
            wrote = n + scales if case["quant"] else n * size
            return {"bytes": n * (size * (2 if case["gate"] else 1) + 2 * stream) + wrote + 4 * c,
                    "flops": n * (16 if case["gate"] else 6)}
        if case["residual"]:   # x, ds and dresidual in the stream's type, dy and dx in io (one where the types agree)
            each = 3 * stream + size * (1 if stream == size else 2)
        else:
            each = size * (5 if case["gate"] else 3)
        return {"bytes": n * each + 8 * c, "flops": n * (30 if case["gate"] else 12)}
    c = case["channels"]
    if op == "step":
        return {"bytes": case["batch"] * c * (4 * size + 8) + 12 * c, "flops": case["batch"] * c * 30}
    n = case["tokens"] * c
    held = -(-case["tokens"] // CHUNK) * c * 4
    if op == "scan":
        state = 2 * case["nseq"] * c * 4 if case["cache"] else 0
        return {"bytes": 4 * n * size + 12 * c + state + (held if case["train"] else 0), "flops": 30 * n}
    return {"bytes": 7 * n * size + held + 24 * c, "flops": 60 * n}


# ---------------------------------------------------------------------------
# exact values: the definitions token by token and row by row, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"scan": _exact_scan, "scan_bwd": _exact_scan_bwd, "step": _exact_step, "norm": _exact_norm,
            "norm_bwd": _exact_norm_bwd}[st["op"]](st)


def _token64(st, at):
    """x, rho, iota, a and the input's weight of the tokens `at`."""
    r = st["r"][at].double() + st["r_bias"].double()
    i = st["i"][at].double() + st["i_bias"].double()
    rho, iota = torch.sigmoid(r), torch.sigmoid(i)
    log_a = st["A"].double() * rho
    a = torch.exp(log_a)
    return st["x"][at].double(), rho, iota, a, (-torch.expm1(log_a) * (1.0 + a)).sqrt()


def _alive(st):
    """For every step of the longest sequence: the sequences that have it, and
    their tokens."""
    edges = st["cu"].tolist()
    lens = [b - a for a, b in zip(edges, edges[1:])]
    order = sorted(range(len(lens)), key=lambda s: -lens[s])
    dev = st["cu"].device
    order_t, first = torch.tensor(order, device=dev), torch.tensor([edges[s] for s in order], device=dev)
    n = len(order)
    for t in range(max(lens)):
        while n and lens[order[n - 1]] <= t:
            n -= 1
        yield t, order_t[:n], first[:n] + t


def _exact_scan(st):
    t, c = st["x"].shape
    s = st["cu"].numel() - 1
    dev = st["x"].device
    state = torch.zeros(s, c, dtype=torch.float64, device=dev)
    if st["state"] is not None:
        old = st["state"].double()
        for k in range(s):
            if int(st["seen"][k]) > 0:
                state[k] = old[int(st["slots"][k])]
    out = torch.zeros(t, c, dtype=torch.float64, device=dev)
    r = {"out": out}
    if st["held"] is not None:
        r["held"] = torch.zeros(st["held"].shape, dtype=torch.float64, device=dev)
    alive = torch.zeros(s, dtype=torch.bool, device=dev)
    for _, seqs, at in _alive(st):
        x, rho, iota, a, m = _token64(st, at)
        h = state[seqs]
        if st["held"] is not None:
            kept = at % CHUNK == 0
            r["held"].index_add_(0, torch.div(at, CHUNK, rounding_mode="floor"), h * kept[:, None])
        h = a * h + m * iota * x
        state[seqs] = h
        out[at] = h
        alive[seqs] = True
    if st["state"] is not None:
        r["state"] = st["state"].double()
        for k in range(s):
            if bool(alive[k]):
                r["state"][int(st["slots"][k])] = state[k]
    return r


def _exact_scan_bwd(st):
    t, c = st["x"].shape
    dev = st["x"].device
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=dev)  # noqa: E731
    before = zeros(t, c)
    state = zeros(st["cu"].numel() - 1, c)
    steps = list(_alive(st))
    for _, seqs, at in steps:
        x, rho, iota, a, m = _token64(st, at)
        before[at] = state[seqs]
        state[seqs] = a * state[seqs] + m * iota * x
    dx, dr, di = zeros(t, c), zeros(t, c), zeros(t, c)
    d_a = zeros(c)
    come = zeros(st["cu"].numel() - 1, c)   # what the later tokens give to the state
    for _, seqs, at in reversed(steps):
        x, rho, iota, a, m = _token64(st, at)
        adj = st["dout"][at].double() + come[seqs]
        come[seqs] = a * adj
        d_log = adj * (before[at] * a - iota * x * a * a / m)
        dx[at] = adj * m * iota
        di[at] = adj * m * x * iota * (1.0 - iota)
        dr[at] = d_log * st["A"].double() * rho * (1.0 - rho)
        d_a += (d_log * rho).sum(0)
    return {"dx": dx, "dr": dr, "di": di, "dA": d_a, "dr_bias": dr.sum(0), "di_bias": di.sum(0)}


def _exact_step(st):
    x, rho, iota, a, m = _token64(st, slice(None))
    state = st["state"].double()
    slots = st["slots"].long()
    h = a * torch.where((st["seen"] > 0)[:, None], state[slots], torch.zeros_like(a)) + m * iota * x
    state[slots] = h
    return {"out": h, "state": state}


def _exact_norm(st):
    r = {}
    v = st["x"].double()
    if st["residual"] is not None:   # the norm is taken of what the residual stream holds
        r["residual"] = v + st["residual"].double()
        v = r["residual"].to(st["residual"].dtype).double()
    if st["z"] is not None:
        z = st["z"].double()
        v = v * z * torch.sigmoid(z)
    parts = []
    for part, w in zip(v.split(st["group"], 1), st["weight"].double().split(st["group"])):
        parts.append(part * torch.rsqrt(part.square().mean(1, keepdim=True) + EPS) * w)
    y = torch.cat(parts, 1)
    if st["quant"]:
        for part in y.split(BLOCK, 1):
            top = part.abs().amax(1, keepdim=True)
            scale = torch.exp2(torch.ceil(torch.log2((top / E4M3_MAX).clamp(min=2.0 ** -100))))
            # e4m3: three fraction bits, the smallest step 2^-9
            u = part / scale
            step = torch.exp2((torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -9))) - 3.0).clamp(min=-9.0))
            part.copy_(torch.round(u / step) * step * scale)
    r["out"] = y
    return r


def _exact_norm_bwd(st):
    x, dy, w, n = st["x"].double(), st["dy"].double(), st["weight"].double(), st["group"]
    z = None if st["z"] is None else st["z"].double()
    dx, dz, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    for lo in range(0, x.shape[1], n):
        cols = slice(lo, lo + n)
        v = x[:, cols] if z is None else x[:, cols] * z[:, cols] * torch.sigmoid(z[:, cols])
        inv = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
        g = dy[:, cols] * w[cols]
        dw[cols] = (dy[:, cols] * v * inv).sum(0)
        dv = inv * g - v * inv ** 3 * (g * v).mean(1, keepdim=True)
        if z is None:
            dx[:, cols] = dv
        else:
            s = torch.sigmoid(z[:, cols])
            dx[:, cols] = dv * z[:, cols] * s
            dz[:, cols] = dv * x[:, cols] * (s + z[:, cols] * s * (1.0 - s))
    r = {"dweight": dw}
    if z is not None:
        r["dz"] = dz
    if st["ds"] is not None:
        dx = dx + st["ds"].double()
        if st["ds"].dtype != st["dy"].dtype:
            r["dresidual"] = dx
    r["dx"] = dx
    return r
