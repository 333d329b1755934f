"""Workloads of the state-cache operators and of the packed prefill, with their plain forms.

Four operators of a serving program that keeps one recurrent state per
sequence, quantized, in a pool of slots:

  write    quantize n sequences' states into their slots
  read     n slots' states back as values
  step     one token for n of the slots: q, k, v in the activations' type,
           q and k heads shared by several value heads
  prefill  packed prompts of unequal lengths: linear attention with a decay
           for each head, from an initial state to a final one

`run` computes them from elementary torch operations, or, where `own` is
true, calls the library.  Both take the same buffers.

Codes are whole numbers that follow from the state by a definition that is
exact to the last bit (include/qstate.h): the plain forms evaluate it in the
order it gives, with its roundings to 32 bits written out and the fused
products formed in 64 bits, because a value next to a border between two
codes would fall on the wrong side otherwise.  INT8 codes are returned as
the integers they are; INT4 codes, two in each byte, as the values that the
read operator gives back.
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _write(n, heads, dk, dv, bits, group, dtype, slots):
    return dict(op="write", n=n, heads=heads, dk=dk, dv=dv, bits=bits, group=group, dtype=dtype, slots=slots)


def _read(n, heads, dk, dv, bits, group, dtype, slots):
    return dict(_write(n, heads, dk, dv, bits, group, dtype, slots), op="read")


def _step(n, heads, qk_heads, dk, dv, bits, group, delta, decay, policy, rounding, dtype, slots):
    return dict(op="step", n=n, heads=heads, qk_heads=qk_heads, dk=dk, dv=dv, bits=bits, group=group,
                delta=delta, decay=decay, policy=policy, rounding=rounding, dtype=dtype, slots=slots)


def _prefill(n, tokens, spread, heads, qk_heads, dk, dv, dtype, initial):
    return dict(op="prefill", n=n, tokens=tokens, spread=spread, heads=heads, qk_heads=qk_heads, dk=dk, dv=dv,
                dtype=dtype, initial=initial)


def listed():
    return [
        # one new sequence of a small model enters the cache: a call's latency
        dict(_write(1, 16, 64, 64, 8, 64, "fp32", 5), name="write_one_int8"),
        # a full batch of prompts ends at once, states in 32 bits as a prefill leaves them
        dict(_write(256, 16, 128, 128, 8, 32, "fp32", 300), name="write_batch_int8"),
        # sequences parked and taken up again in 16 bits, INT4 between: write, then read back
        dict(_write(100, 24, 128, 80, 4, 32, "bf16", 131), name="park_and_resume_int4"),
        # states of many slots back in 32 bits, for another chunk of their prompts
        dict(_read(256, 16, 128, 128, 4, 64, "fp32", 300), name="read_batch_int4"),
        # one user, small gated delta-rule model, one token: latency
        dict(_step(1, 4, 4, 64, 64, 8, 64, 1, "scalar", "persistent", "nearest", "bf16", 3), name="step_one_int8"),
        # gated delta-rule layer, 64 sequences, INT4 with directional rounding, q/k heads shared by two
        # value heads; the new states are read back (a draft token's snapshot)
        dict(_step(64, 16, 8, 128, 128, 4, 32, 1, "scalar", "persistent", "bdr", "bf16", 80), name="step_snapshot_int4"),
        # scalar-decay linear write, all heads on one q/k head
        dict(_step(256, 64, 1, 128, 64, 8, 64, 0, "scalar", "persistent", "nearest", "fp16", 256),
             name="step_linear_int8"),
        # the largest batch, dynamic scales
        dict(_step(768, 16, 16, 128, 128, 8, 32, 1, "scalar", "dynamic", "nearest", "bf16", 800),
             name="step_large_int8"),
        # a short follow-up of one user: latency
        dict(_prefill(1, 17, 0.0, 8, 8, 64, 64, "bf16", True), name="prefill_short"),
        # one long prompt: few heads to spread over the card
        dict(_prefill(1, 16384, 0.0, 16, 16, 128, 128, "bf16", False), name="prefill_long"),
        # a scheduler's batch: unequal lengths, continued and new, shared q/k heads
        dict(_prefill(32, 12000, 1.0, 64, 8, 128, 64, "fp16", True), name="prefill_ragged"),
        # equal prompts, every head its own q and k
        dict(_prefill(64, 16384, 0.0, 16, 16, 128, 128, "bf16", True), name="prefill_batch"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "step", "prefill"])
    dk = rng.choice([64, 128])
    dv = 16 * _log(rng, 2, 12)
    heads = rng.choice([1, 2, 4, 6, 8, 12, 16, 24, 32, 64])
    dtype = rng.choice(["fp32", "fp16", "bf16"])
    bits = rng.choice([4, 8])
    group = rng.choice([g for g in (32, 64, 128) if g <= dk])
    # states of a batch: at most 48 M elements, the large listed cases have 67 M and more
    most = max(1, 48_000_000 // (heads * dk * dv))
    if op in ("write", "read"):
        n = _log(rng, 1, min(400, most))
        make = _write if op == "write" else _read
        return make(n, heads, dk, dv, bits, group, dtype, n + rng.randrange(0, 40))
    qk = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
    if op == "step":
        n = _log(rng, 1, min(800, most))
        return _step(n, heads, qk, dk, dv, bits, group, rng.choice([0, 1]), rng.choice(["scalar", "scalar", "diagonal"]),
                     rng.choice(["dynamic", "persistent"]), rng.choice(["nearest", "bdr"]), dtype,
                     n + rng.randrange(0, 40))
    # at most 4 G state updates (tokens x heads x dk x dv); the listed long prompt has 4.3 G
    n = _log(rng, 1, 48)
    tokens = _log(rng, n, max(n + 1, min(16000, 4_000_000_000 // (heads * dk * dv))))
    return _prefill(n, tokens, rng.choice([0.0, 0.5, 1.0]), heads, qk, dk, dv, rng.choice(["fp16", "bf16"]),
                    rng.choice([True, False]))


def _lengths(case):
    """Lengths of the case's prompts, from the case alone: even, or uneven by `spread` (empty ones among them)."""
    n, tokens = case["n"], case["tokens"]
    rng = random.Random(1000003 * n + tokens)
    w = [math.exp(rng.gauss(0.0, case["spread"])) for _ in range(n)]
    cut = [0]
    for x in w:
        cut.append(cut[-1] + x)
    at = [round(tokens * c / cut[-1]) for c in cut]
    at[-1] = tokens
    return [b - a for a, b in zip(at, at[1:])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _gates(gen, law, *shape):
    """Decays and write strengths: slow sigmoid gates (delta rule, diagonal), or the steps of a scalar-decay model."""
    x, y = _normal(gen, *shape), _normal(gen, *shape[:2])
    if law == "linear":
        return torch.exp(-torch.nn.functional.softplus(x) * 0.1), torch.nn.functional.softplus(y)
    return torch.sigmoid(3.0 + x), torch.sigmoid(y)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * seed + 17)
    c, T = case, TYPES[case["dtype"]]
    n, H, dk, dv = c["n"], c["heads"], c["dk"], c["dv"]
    st = {"case": dict(case)}
    if c["op"] == "prefill":
        N, Hk = c["tokens"], c["qk_heads"]
        lens = _lengths(c)
        starts = [0]
        for x in lens:
            starts.append(starts[-1] + x)
        st["lens"] = lens
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["q"] = _normal(gen, N, Hk, dk, std=dk ** -0.5, dtype=T)
        st["k"] = _unit(_normal(gen, N, Hk, dk)).to(T)
        st["v"] = _normal(gen, N, H, dv, dtype=T)
        st["alpha"], st["beta"] = _gates(gen, "linear", N, H)
        st["S0"] = _normal(gen, n, H, dv, dk, std=0.5) if c["initial"] else None
        st["S"] = torch.empty(n, H, dv, dk, device="cuda")
        st["o"] = torch.empty(N, H, dv, dtype=T, device="cuda")
        return st
    # a pool that holds every slot's state, and the slots of this call in no order
    pool = c["slots"]
    st["codes"] = torch.zeros(pool, H, dv, dk * c["bits"] // 8, dtype=torch.uint8, device="cuda")
    st["scales"] = torch.zeros(pool, H, dv, dk // c["group"], device="cuda")
    st["slots"] = torch.randperm(pool, generator=gen, device="cuda")[:n].to(torch.int32)
    every = torch.arange(pool, dtype=torch.int32, device="cuda")
    if c["op"] == "write":
        st["S"] = _normal(gen, n, H, dv, dk, std=dk ** -0.5, dtype=T)
        st["back"] = torch.empty_like(st["S"]) if c["bits"] == 4 else None
        return st
    _plain_write(c, _normal(gen, pool, H, dv, dk, std=dk ** -0.5), every, st["codes"], st["scales"])
    if c["op"] == "read":
        st["back"] = torch.empty(n, H, dv, dk, dtype=T, device="cuda")
        return st
    Hk = c["qk_heads"]
    st["q"] = _normal(gen, n, Hk, dk, dtype=T)
    st["k"] = _unit(_normal(gen, n, Hk, dk)).to(T)
    st["v"] = _normal(gen, n, H, dv, dtype=T)
    law = "linear" if not c["delta"] and c["decay"] == "scalar" else "gate"
    st["alpha"], st["beta"] = _gates(gen, law, n, H, *([dk] if c["decay"] == "diagonal" else []))
    st["o"] = torch.empty(n, H, dv, dtype=T, device="cuda")
    st["back"] = torch.empty(n, H, dv, dk, dtype=torch.bfloat16, device="cuda") if c["bits"] == 4 else None
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _unpack(codes, bits):
    if bits == 8:
        return codes.view(torch.int8).float()
    pair = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    return ((pair ^ 8).to(torch.int8) - 8).float()


def _pack(c, bits):
    c = c.to(torch.int8).view(torch.uint8)
    return c if bits == 8 else (c[..., 0::2] & 15) | (c[..., 1::2] << 4)


def _nearest(x, scale, qmax):
    """The integers nearest to x / scale, by the definition's reciprocal of the scale; 0 where the scale is 0."""
    inv = torch.where(scale > 0, scale.reciprocal(), 0.0)
    return torch.round(x.double() * inv.double()).clamp(-qmax, qmax).float()


def _plain_write(c, S, slots, codes, scales):
    qmax = 7.0 if c["bits"] == 4 else 127.0
    x = S.float().unflatten(-1, (-1, c["group"]))
    s = x.abs().amax(-1) / torch.full((), qmax, device=S.device)
    at = slots.long()
    codes[at] = _pack(_nearest(x, s[..., None], qmax).flatten(-2), c["bits"])
    scales[at] = s


def _plain_read(c, slots, codes, scales):
    at = slots.long()
    d = _unpack(codes[at], c["bits"]).unflatten(-1, (-1, c["group"])) * scales[at][..., None]
    return d.flatten(-2)


def _fma(a, b, c):
    return (a.double() * b.double() + c.double()).float()


def _dot(a, b):
    """a . b over the last axis in the definition's order: eight chains for each 32 columns, then pairwise."""
    a, b = a.unflatten(-1, (-1, 4, 8)), b.unflatten(-1, (-1, 4, 8))
    p = a[..., 0, :] * b[..., 0, :]
    p = _fma(a[..., 1, :], b[..., 1, :], p)
    p = _fma(a[..., 2, :], b[..., 2, :], p)
    p = _fma(a[..., 3, :], b[..., 3, :], p)
    p = (p[..., 0:2] + p[..., 4:6]) + (p[..., 2:4] + p[..., 6:8])
    t = p[..., 0] + p[..., 1]
    t = t[..., 0::2] + t[..., 1::2]
    return (t[..., 0::2] + t[..., 1::2] if t.shape[-1] > 1 else t)[..., 0]


def _plain_step(st):
    c, at = st["case"], st["slots"].long()
    share = c["heads"] // c["qk_heads"]
    qmax = 7.0 if c["bits"] == 4 else 127.0
    grouped = lambda x: x.unflatten(-1, (-1, c["group"]))
    q, k = (st[x].float().repeat_interleave(share, 1)[:, :, None, :] for x in ("q", "k"))
    v, beta, alpha = st["v"].float(), st["beta"][..., None], st["alpha"]
    alpha = alpha[:, :, None, None] if alpha.dim() == 2 else alpha[:, :, None, :]
    code, s = _unpack(st["codes"][at], c["bits"]), st["scales"][at]
    per_column = s.repeat_interleave(c["group"], -1)
    Sd = code * (per_column * alpha)
    w = beta * (v - _dot(Sd, k.expand_as(Sd))) if c["delta"] else beta * v
    x = _fma(w[..., None], k, Sd)
    o = _dot(x, q.expand_as(x))
    if c["policy"] == "dynamic":
        s = grouped(x).abs().amax(-1) / torch.full((), qmax, device=x.device)
    new = _nearest(grouped(x), s[..., None], qmax).flatten(-2)
    if c["rounding"] == "bdr":
        d, r = code * per_column, new * s.repeat_interleave(c["group"], -1)
        sigma = torch.sign(w)[..., None] * torch.sign(k)
        on = (s > 0).repeat_interleave(c["group"], -1)
        new = new + ((sigma > 0) & (r < d) & on).float() - ((sigma < 0) & (r > d) & on).float()
        new = new.clamp(-qmax, qmax)
    st["codes"][at] = _pack(new, c["bits"])
    st["scales"][at] = s
    return o.to(st["o"].dtype)


def _plain_prefill(st):
    """Chunks of 64 tokens of every prompt side by side; the state before each chunk is a sum over the chunks before it."""
    c, C, dev = st["case"], 64, st["q"].device
    H, Hk, share, n = c["heads"], c["qk_heads"], c["heads"] // c["qk_heads"], c["n"]
    lens = torch.tensor(st["lens"], device=dev)
    starts = lens.cumsum(0) - lens
    count = (lens + C - 1) // C
    seq = torch.repeat_interleave(torch.arange(n, device=dev), count)
    order = torch.arange(len(seq), device=dev) - (count.cumsum(0) - count)[seq]
    at = (starts[seq] + order * C)[:, None] + torch.arange(C, device=dev)
    valid = at < (starts + lens)[seq][:, None]
    at = at.clamp(max=c["tokens"] - 1)
    # running logarithms of the decays over the whole buffer, in 64 bits; only differences within a prompt are used
    logs = st["alpha"].double().log()
    run = logs.cumsum(0)
    before = run - logs
    last = valid.sum(1) - 1
    head = before[at[:, 0]]                                            # [chunks, H]
    tail = run[at[torch.arange(len(seq), device=dev), last]]
    here = run[at].transpose(1, 2)                                     # [chunks, H, C]
    take = lambda x: (x[at].float() * valid[..., None, None]).transpose(1, 2)
    q, k, v = take(st["q"]), take(st["k"]), take(st["v"])              # [chunks, heads, C, dim]
    wide = lambda x: x.repeat_interleave(share, 1)
    beta = (st["beta"][at] * valid[..., None]).transpose(1, 2)
    past = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    decay = torch.where(past, here[..., :, None] - here[..., None, :], -math.inf).exp().float()
    o = (wide(q @ k.transpose(-1, -2)) * decay * beta[..., None, :]) @ v
    left = (tail[..., None] - here).exp().float() * beta
    own_part = (v * left[..., None]).transpose(-1, -2) @ wide(k)       # [chunks, H, dv, dk]
    same = seq[:, None] == seq[None, :]
    earlier = same & (order[:, None] > order[None, :])
    weight = torch.where(earlier[..., None], head[:, None] - tail[None, :], -math.inf).exp().float()
    flat = own_part.flatten(2).transpose(0, 1)                         # [H, chunks, dv * dk]
    S_in = weight.permute(2, 0, 1) @ flat
    whole = torch.zeros(n, H, dtype=torch.float64, device=dev).index_add_(0, torch.repeat_interleave(
        torch.arange(n, device=dev), lens), logs)
    first = starts[seq].clamp(max=c["tokens"] - 1)
    member = torch.arange(n, device=dev)[:, None] == seq[None, :]
    end = before[starts.clamp(max=c["tokens"] - 1)] + whole
    to_end = torch.where(member[..., None], end[:, None] - tail[None, :], -math.inf).exp().float()
    S = (to_end.permute(2, 0, 1) @ flat).transpose(0, 1).unflatten(-1, (c["dv"], c["dk"]))
    S_in = S_in.transpose(0, 1).unflatten(-1, (c["dv"], c["dk"]))
    if st["S0"] is not None:
        S_in = S_in + (head - before[first]).exp().float()[..., None, None] * st["S0"][seq]
        S = S + whole.exp().float()[..., None, None] * st["S0"]
    o = o + (wide(q) @ S_in.transpose(-1, -2)) * (here - head[..., None]).exp().float()[..., None]
    out = torch.empty(c["tokens"], H, c["dv"], device=dev)
    out[at[valid]] = o.transpose(1, 2)[valid]
    return out.to(st["o"].dtype), S


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _handle(st):
    """The cache or prefill object that a user's program makes once and keeps."""
    if "handle" not in st:
        from ssm_decode_step_b200 import Config, PackedPrefill, StateCache
        c = st["case"]
        if c["op"] == "prefill":
            st["handle"] = PackedPrefill(Config(0, c["dk"], c["dv"], 8, 32, 0), c["heads"], c["qk_heads"],
                                         max_tokens=c["tokens"], max_sequences=c["n"])
        else:
            cfg = Config(c["slots"] * c["heads"], c["dk"], c["dv"], c["bits"], c["group"], c.get("delta", 0),
                         c.get("decay", "scalar"), c.get("policy", "dynamic"), c.get("rounding", "nearest"))
            st["handle"] = StateCache(cfg, c["heads"], codes=st["codes"], scales=st["scales"])
    return st["handle"]


def run(state):
    st, op = state, state["case"]["op"]
    c = st["case"]
    if op == "prefill":
        if own:
            _handle(st).run(st["starts"], st["q"], st["k"], st["v"], st["alpha"], st["beta"], S0=st["S0"], S=st["S"],
                            o=st["o"])
            return {"o": st["o"], "S": st["S"]}
        o, S = _plain_prefill(st)
        return {"o": o, "S": S}
    if op == "read":
        if own:
            _handle(st).read(st["slots"], st["back"])
            return {"values": st["back"]}
        return {"values": _plain_read(c, st["slots"], st["codes"], st["scales"]).to(st["back"].dtype)}
    out = {}
    if op == "write":
        if own:
            _handle(st).write(st["slots"], st["S"])
        else:
            _plain_write(c, st["S"], st["slots"], st["codes"], st["scales"])
    elif own:
        _handle(st).step(st["slots"], st["q"], st["k"], st["v"], st["alpha"], st["beta"], o=st["o"])
        out["o"] = st["o"]
    else:
        out["o"] = _plain_step(st)
    if c["bits"] == 8:
        out["codes"] = st["codes"].view(torch.int8)
    elif own:
        _handle(st).read(st["slots"], st["back"])
        out["values"] = st["back"]
    else:
        out["values"] = _plain_read(c, st["slots"], st["codes"], st["scales"]).to(st["back"].dtype)
    out["scales"] = st["scales"]
    return out


def work(case):
    c = case
    n, H, dk, dv, e = c["n"], c["heads"], c["dk"], c["dv"], TYPES[c["dtype"]].itemsize
    if c["op"] == "prefill":
        N = c["tokens"]
        per_token = 2 * c["qk_heads"] * dk * e + 2 * H * dv * e + 8 * H
        return {"bytes": N * per_token + (2 if c["initial"] else 1) * n * H * dv * dk * 4 + 4 * (n + 1),
                "flops": 4.0 * N * H * dk * dv}
    elements = n * H * dk * dv
    codes, scales = elements * c["bits"] / 8, elements / c["group"] * 4
    if c["op"] in ("write", "read"):
        back = elements * e + codes + scales if c["op"] == "write" and c["bits"] == 4 else 0
        return {"bytes": codes + scales + elements * e + back, "flops": 3.0 * elements}
    vectors = n * (2 * c["qk_heads"] * dk + 2 * H * dv) * e + n * H * 4 * (dk + 1 if c["decay"] == "diagonal" else 2)
    back = elements * 2 + codes + scales if c["bits"] == 4 else 0
    return {"bytes": 2 * codes + (2 if c["policy"] == "dynamic" else 1) * scales + vectors + back,
            "flops": (8.0 if c["delta"] else 6.0) * elements}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    c, n = case, case["n"]
    H, dk, dv = c["heads"], c["dk"], c["dv"]
    if c["op"] == "prefill":
        return _exact_prefill(st)
    rows = st["slots"].long()
    qmax = 7 if c["bits"] == 4 else 127

    def values(of):
        raw = of["codes"][rows].to(torch.int16)
        if c["bits"] == 8:
            code = torch.where(raw > 127, raw - 256, raw)
        else:
            low, high = raw % 16, raw // 16
            code = torch.empty(n, H, dv, dk, dtype=torch.int16, device=raw.device)
            code[..., 0::2], code[..., 1::2] = low, high
            code = torch.where(code > 7, code - 16, code)
        return (code.double().view(n, H, dv, -1, c["group"]) * of["scales"][rows].double().unsqueeze(-1)).view(n, H, dv, dk)

    def quantized(x, scale=None):
        g = x.view(n, H, dv, -1, c["group"])
        if scale is None:
            scale = g.abs().max(-1).values / qmax
        # the definition's reciprocal is that of the 32-bit scale, itself rounded to 32 bits: with states in 16 bits,
        # half a group's largest value lies on a border between two codes, and those roundings decide
        stored = scale.float()
        inverse = torch.where(stored == 0, 0.0, 1.0 / stored).double()
        return torch.round(g * inverse.unsqueeze(-1)).clamp(-qmax, qmax), scale

    if c["op"] == "read":
        return {"values": values(st)}
    if c["op"] == "write":
        code, scale = quantized(st["S"].double())
    else:
        d = values(st)
        spread = torch.arange(H, device=d.device) // (H // c["qk_heads"])
        q, k = st["q"].double()[:, spread], st["k"].double()[:, spread]
        a = st["alpha"].double()
        x = d * (a.view(n, H, 1, 1) if a.dim() == 2 else a.view(n, H, 1, dk))
        w = st["v"].double()
        if c["delta"]:
            w = w - torch.einsum("nhij,nhj->nhi", x, k)
        w = w * st["beta"].double().unsqueeze(-1)
        x = x + torch.einsum("nhi,nhj->nhij", w, k)
        o = torch.einsum("nhij,nhj->nhi", x, q)
        kept = st["scales"][rows].double() if c["policy"] == "persistent" else None
        code, scale = quantized(x, kept)
        if c["rounding"] == "bdr":
            way = (torch.sign(w).unsqueeze(-1) * torch.sign(k).unsqueeze(-2)).view_as(code)
            off = code * scale.unsqueeze(-1) - d.view_as(code)
            # a product that equals the stored element in 64 bits, but for their last places, has not moved
            moved = off.abs() > 1e-12 * d.view_as(code).abs()
            code = (code + (moved & (way * off < 0)) * way).clamp(-qmax, qmax)
    scales = st["scales"].double().clone()
    scales[rows] = scale
    out = {"scales": scales}
    if c["op"] == "step":
        out["o"] = o
    if c["bits"] == 8:
        out["codes"] = None   # whole numbers, some of them next to a border in 32 bits
    else:
        out["values"] = (code * scale.unsqueeze(-1)).view(n, H, dv, dk)
    return out


def _exact_prefill(st):
    """Token by token, all prompts side by side: the n-th token of every prompt at once."""
    c, lens = st["case"], st["lens"]
    n, H, dk, dv = c["n"], c["heads"], c["dk"], c["dv"]
    dev = st["q"].device
    spread = torch.arange(H, device=dev) // (H // c["qk_heads"])
    S = torch.zeros(n, H, dv, dk, dtype=torch.float64, device=dev) if st["S0"] is None else st["S0"].double()
    o = torch.zeros(c["tokens"], H, dv, dtype=torch.float64, device=dev)
    # prompts in falling order of length: the first m of them still have a token
    by_length = sorted(range(n), key=lambda i: -lens[i])
    S = S[torch.tensor(by_length, device=dev)].contiguous()
    starts = st["starts"].long()[:-1][torch.tensor(by_length, device=dev)]
    alive, m = [], n
    for t in range(max(lens)):
        while m and lens[by_length[m - 1]] <= t:
            m -= 1
        alive.append(m)
    for t, m in enumerate(alive):
        row = starts[:m] + t
        k, q = st["k"][row][:, spread].double(), st["q"][row][:, spread].double()
        w = st["v"][row].double() * st["beta"][row].double().unsqueeze(-1)
        S[:m].mul_(st["alpha"][row].double()[..., None, None]).addcmul_(w.unsqueeze(-1), k.unsqueeze(-2))
        o[row] = (S[:m] @ q.unsqueeze(-1)).squeeze(-1)
    final = torch.empty_like(S)
    final[torch.tensor(by_length, device=dev)] = S
    return {"o": o, "S": final}
