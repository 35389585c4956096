"""The operators around a linear-attention state, as a decoder layer runs them:

  prompt  linear attention with a decay for each head over packed prompts
          (S <- a S + v k^T, o = S q), from and into a pool of states;
  token   the same for one token of each sequence;
  rotary  rotary positions on q and k;
  norm    group norm of the heads' outputs with an activation or a gate.

`run` computes an operator in elementary torch operations, or, where `own` is
set, through the package's entry points.  Token-major layouts throughout:
q, k [tokens][Hk][dk], v [tokens][Hv][dv], states [slots][Hv][dv][dk]; value
head h reads key head h / (Hv / Hk)."""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}
CHUNK = 128  # tokens of a chunk in the plain form


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one short question to an idle server: its latency
        dict(name="prompt_one_short", op="prompt", seqs=1, tokens=77, longest=77, hk=16, hv=32, dk=128, dv=128,
             io=BF16, out=BF16, decay="token", fused=True, fresh=True),
        # a batch of prompts of very different lengths, some continuing an earlier state,
        # grouped heads, outputs rounded to the layer's type
        dict(name="prompt_batch", op="prompt", seqs=24, tokens=20011, longest=6000, hk=16, hv=32, dk=128, dv=128,
             io=BF16, out=BF16, decay="token", fused=True, fresh=False),
        # the same kind of batch with fp32 outputs, the library's default, one head per key
        dict(name="prompt_batch_f32_out", op="prompt", seqs=9, tokens=7000, longest=3000, hk=32, hv=32, dk=128,
             dv=128, io=BF16, out=F32, decay="token", fused=False, fresh=False),
        # one long document, fixed decays
        dict(name="prompt_one_long", op="prompt", seqs=1, tokens=32768, longest=32768, hk=32, hv=32, dk=128, dv=128,
             io=BF16, out=BF16, decay="head", fused=False, fresh=True),
        # a small model in fp32 throughout
        dict(name="prompt_f32_small", op="prompt", seqs=5, tokens=3001, longest=1100, hk=2, hv=8, dk=64, dv=64,
             io=F32, out=F32, decay="token", fused=False, fresh=False),
        # decoding for one user
        dict(name="token_one", op="token", seqs=1, hk=16, hv=32, dk=128, dv=128, io=BF16, out=BF16, decay="token",
             fused=True),
        # decoding for a full batch
        dict(name="token_batch", op="token", seqs=256, hk=32, hv=32, dk=128, dv=128, io=BF16, out=F32, decay="head",
             fused=False),
        # q and k of a decoding batch, far positions
        dict(name="rotary_tokens", op="rotary", tokens=64, hq=32, hk=16, d=128, rot=128, layout="half", io=BF16,
             scaling="none", far=1 << 20, inverse=False, fused=True),
        # q and k of a long prompt, a quarter-to-half of the head rotated, context extended
        dict(name="rotary_prompt", op="rotary", tokens=16381, hq=32, hk=32, d=128, rot=64, layout="interleaved",
             io=BF16, scaling="parts", far=1 << 17, inverse=False, fused=False),
        # a decoding batch's head outputs, gated
        dict(name="norm_tokens", op="norm", tokens=64, groups=32, size=128, kind="rms", act="silu", gate="after",
             weight="group", bias=False, io=BF16, out=BF16),
        # a long prompt's head outputs, fp32 as the prompt operator leaves them
        dict(name="norm_prompt", op="norm", tokens=16384, groups=32, size=128, kind="mean", act="silu", gate="none",
             weight="channel", bias=True, io=F32, out=BF16),
        # an odd group size, gated before the norm
        dict(name="norm_odd", op="norm", tokens=4099, groups=7, size=100, kind="rms", act="sigmoid", gate="before",
             weight="channel", bias=False, io=F32, out=F32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _any(rng)
    while work(c)["bytes"] > 6e8:
        c["tokens" if "tokens" in c else "seqs"] //= 2
        if "longest" in c:
            c["longest"] = c["longest"] // 2 + 1
    return c


def _any(rng):
    op = rng.choice(["prompt", "prompt", "token", "rotary", "norm"])
    if op in ("prompt", "token"):
        io = rng.choice([BF16, BF16, BF16, F32])
        d = rng.choice([32, 64, 128, 128, 128])
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        c = dict(op=op, seqs=_log_int(rng, 1, 32 if op == "prompt" else 256), hk=hk,
                 hv=hk * rng.choice([1, 1, 2, 4] if hk < 16 else [1, 2]), dk=d,
                 dv=rng.choice([d, d, d, 32, 64, 128]), io=io, out=io if io == F32 else rng.choice([BF16, F32]),
                 decay=rng.choice(["token", "token", "head"]), fused=rng.random() < 0.5)
        if op == "prompt":
            c["tokens"] = max(c["seqs"], _log_int(rng, 1, 16384))
            c["longest"] = max(-(-c["tokens"] // c["seqs"]), int(c["tokens"] * rng.uniform(0.2, 1.0)))
            c["fresh"] = rng.random() < 0.5
        return c
    if op == "rotary":
        d = rng.choice([32, 64, 80, 128, 256])
        return dict(op=op, tokens=_log_int(rng, 1, 16384), hq=rng.choice([1, 4, 7, 16, 32]),
                    hk=rng.choice([1, 1, 4, 8, 16]), d=d, rot=rng.choice([d, d, d // 2, d // 4 * 2 - 2]),
                    layout=rng.choice(["half", "interleaved"]), io=rng.choice([BF16, BF16, F32]),
                    scaling=rng.choice(["none", "linear", "ntk", "parts"]), far=_log_int(rng, 64, 1 << 21),
                    inverse=rng.random() < 0.25, fused=rng.random() < 0.5)
    gate = rng.choice(["none", "after", "before"])
    io = rng.choice([BF16, BF16, F32])
    return dict(op=op, tokens=_log_int(rng, 1, 16384), groups=rng.choice([1, 3, 8, 16, 32]),
                size=rng.choice([16, 32, 64, 100, 128, 128, 256, 333]), kind=rng.choice(["rms", "mean"]),
                act=rng.choice(["none", "silu", "sigmoid"]), gate=gate,
                weight=rng.choice(["none", "group", "channel"]), bias=rng.random() < 0.3, io=io,
                out=rng.choice([io, F32]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _lengths(case, gen):
    """`seqs` lengths that add up to `tokens`, none above `longest`; from four
    sequences on the second is empty."""
    n, total, top = case["seqs"], case["tokens"], case["longest"]
    share = torch.exp(torch.randn(n, generator=gen, dtype=torch.float64))
    share[0] = share.max() * 4
    if n >= 4:
        share[1] = 0.0
    x = torch.clamp((share / share.sum() * total).floor().long(), max=top)
    for i in range(n):  # what the floor and the bound left over, to the first with room
        if not (n >= 4 and i == 1):
            x[i] += min(top - int(x[i]), total - int(x.sum()))
    if int(x.sum()) < total:
        x[1] += total - int(x.sum())
    return x


def _unit(x):
    return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True).clamp_min(1e-6)


def _qkv(case, tokens, rnd):
    """q, k unit vectors per head, v normal; apart, or as slices of one fused
    projection's rows."""
    hk, hv, dk, dv, dt = case["hk"], case["hv"], case["dk"], case["dv"], DT[case["io"]]
    q, k, v = _unit(rnd(tokens, hk, dk)).to(dt), _unit(rnd(tokens, hk, dk)).to(dt), rnd(tokens, hv, dv).to(dt)
    if not case["fused"]:
        return q, k, v
    a, b = hk * dk, hv * dv
    rows = torch.cat([q.reshape(tokens, a), k.reshape(tokens, a), v.reshape(tokens, b)], dim=1)
    return (rows[:, :a].unflatten(1, (hk, dk)), rows[:, a:2 * a].unflatten(1, (hk, dk)),
            rows[:, 2 * a:].unflatten(1, (hv, dv)))


def _decay(case, tokens, gen):
    hv = case["hv"]
    if case["decay"] == "token":  # data-dependent gates, as the library's workloads draw them
        return 0.9 + 0.1 * torch.rand((tokens, hv), generator=gen, device="cuda")
    h = torch.arange(1, hv + 1, device="cuda", dtype=torch.float64)  # fixed slopes, fast to slow heads
    return torch.exp(-torch.exp2(-8.0 * h / hv)).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))

    def rnd(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] in ("prompt", "token"):
        n = case["seqs"]
        tokens = case["tokens"] if case["op"] == "prompt" else n
        s["q"], s["k"], s["v"] = _qkv(case, tokens, rnd)
        s["decay"] = _decay(case, tokens, gen)
        slots = n + 3  # a pool with a few states of other sequences
        s["S"] = 0.1 * rnd(slots, case["hv"], case["dv"], case["dk"])
        s["slots"] = torch.randperm(slots, generator=host)[:n].to(torch.int32).cuda()
        s["out"] = torch.empty((tokens, case["hv"], case["dv"]), dtype=DT[case["out"]], device="cuda")
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "prompt":
            lengths = _lengths(case, host)
            s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), lengths.cumsum(0)]).to(torch.int32).cuda()
            fresh = torch.ones(n) if case["fresh"] else torch.arange(n) % 3 == 0
            s["fresh"] = fresh.to(torch.int32).cuda()
    elif case["op"] == "rotary":
        n, hq, hk, d, dt = case["tokens"], case["hq"], case["hk"], case["d"], DT[case["io"]]
        s["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        if case["fused"]:
            rows = rnd(n, (hq + hk) * d).to(dt)
            s["q"], s["k"] = rows[:, :hq * d].unflatten(1, (hq, d)), rows[:, hq * d:].unflatten(1, (hk, d))
        else:
            s["q"], s["k"] = rnd(n, hq, d).to(dt), rnd(n, hk, d).to(dt)
        s["q_out"] = torch.empty((n, hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((n, hk, d), dtype=dt, device="cuda")
        freq, s["magnitude"] = _frequencies(case)
        s["freq"] = freq.cuda()
    else:
        n, g, d, dt = case["tokens"], case["groups"], case["size"], DT[case["io"]]
        s["x"] = (rnd(n, g, d) * torch.exp(rnd(n, g, 1)) + 0.3).to(dt)
        s["z"] = rnd(n, g, d).to(dt) if case["gate"] != "none" else None
        wide = {"none": None, "group": (d,), "channel": (g, d)}[case["weight"]]
        s["w"] = 1.0 + 0.2 * rnd(*wide) if wide else None
        s["b"] = 0.1 * rnd(g, d) if case["bias"] else None
        s["out"] = torch.empty((n, g, d), dtype=DT[case["out"]], device="cuda")
    return s


# Rotary frequencies: theta^(-2i/rot), scaled for a context 8 times the trained one.
THETA, FACTOR, TRAINED, FAST, SLOW = 10000.0, 8.0, 8192.0, 32.0, 1.0


def _frequencies(case):
    """([rot / 2] angles per position in 64 bits, the factor on cos and sin)."""
    rot, kind = case["rot"], case["scaling"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = THETA ** (-2.0 * i / rot)
    if kind == "linear":
        return f / FACTOR, 1.0
    if kind == "ntk":
        return (THETA * FACTOR ** (rot / max(rot - 2, 1))) ** (-2.0 * i / rot), 1.0
    if kind == "parts":  # few turns within the trained context: interpolated; many: kept
        turns = TRAINED * f / (2 * math.pi)
        keep = ((turns - SLOW) / (FAST - SLOW)).clamp(0.0, 1.0)
        return f * keep + f / FACTOR * (1.0 - keep), 0.1 * math.log(FACTOR) + 1.0
    return f, 1.0


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _rows_of(case, t):
    """[.., Hk, d] -> [.., Hv, d] in fp32."""
    return t.float().repeat_interleave(case["hv"] // case["hk"], dim=-2)


def _plain_prompt(s):
    c = s["case"]
    off = s["offsets"].long()
    lengths = off[1:] - off[:-1]
    n, hv, dk, dv = c["seqs"], c["hv"], c["dk"], c["dv"]
    # every sequence cut into chunks: rows of tokens, with -1 past its end
    chunks = (lengths + CHUNK - 1) // CHUNK
    bound = -(-c["tokens"] // CHUNK) + n
    first = torch.cumsum(chunks, 0) - chunks
    at = torch.arange(bound, device="cuda")
    seq = torch.searchsorted(torch.cumsum(chunks, 0), at, right=True).clamp(max=n - 1)
    live = at < chunks.sum()
    row = (at - first[seq])[:, None] * CHUNK + torch.arange(CHUNK, device="cuda")
    valid = live[:, None] & (row < lengths[seq][:, None])
    token = torch.where(valid, off[seq][:, None] + row, 0).clamp(max=max(c["tokens"] - 1, 0))
    q = _rows_of(c, s["q"][token])                                     # [chunks][C][Hv][dk]
    k = torch.where(valid[..., None, None], _rows_of(c, s["k"][token]), 0.0)
    v = torch.where(valid[..., None, None], s["v"][token].float(), 0.0)
    la = torch.log(s["decay"].double())
    la = la[token] if c["decay"] == "token" else la.expand(bound, CHUNK, hv)
    la = torch.where(valid[..., None], la, 0.0).transpose(1, 2)         # [chunks][Hv][C]
    cum = torch.cumsum(la, -1)
    q, k, v = (x.transpose(1, 2) for x in (q, k, v))                    # [chunks][Hv][C][d]
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    gap = torch.where(lower, cum[..., :, None] - cum[..., None, :], -math.inf)
    inner = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * torch.exp(gap).float(), v)
    left = torch.exp(cum[..., -1:] - cum).float()
    grown = torch.matmul(v.transpose(-1, -2), k * left[..., None])      # [chunks][Hv][dv][dk]
    # the state before a chunk: all earlier chunks of its sequence, decayed, and the first state
    total = torch.cumsum(cum[..., -1], 0)                               # [chunks][Hv]
    before = total - cum[..., -1]
    same = (seq[:, None] == seq[None, :]) & live[None, :] & (at[:, None] > at[None, :])
    far = torch.where(same[..., None], before[:, None] - total[None, :], -math.inf)
    fade = torch.exp(far).float().permute(2, 0, 1)                      # [Hv][chunks][chunks]
    base = torch.matmul(fade, grown.transpose(0, 1).flatten(2)).unflatten(2, (dv, dk)).transpose(0, 1)
    slot = s["slots"].long()
    start = torch.where(s["fresh"].bool()[:, None, None, None], 0.0, s["S"][slot])
    head = before[first.clamp(max=bound - 1)]                           # [seqs][Hv]
    base = base + torch.exp(before - head[seq]).float()[..., None, None] * start[seq]
    o = inner + torch.exp(cum).float()[..., None] * torch.matmul(q, base.transpose(-1, -2))
    out = torch.zeros((c["tokens"], hv, dv), dtype=DT[c["out"]], device="cuda")
    out[token[valid]] = o.transpose(1, 2)[valid].to(out.dtype)
    last = (first + chunks - 1).clamp(min=0)
    end = torch.exp(cum[last, :, -1]).float()[..., None, None] * base[last] + grown[last]
    s["S"][slot] = torch.where((chunks > 0)[:, None, None, None], end, start)
    return out, s["S"]


def _plain_token(s):
    c = s["case"]
    q, k, v = _rows_of(c, s["q"]), _rows_of(c, s["k"]), s["v"].float()
    slot = s["slots"].long()
    a = s["decay"].expand(c["seqs"], c["hv"])[..., None, None]
    S = a * s["S"][slot] + v[..., None] * k[..., None, :]
    s["S"][slot] = S
    return (S * q[..., None, :]).sum(-1).to(DT[c["out"]]), s["S"]


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"]
    sign = -1.0 if c["inverse"] else 1.0
    cos = (torch.cos(angle) * s["magnitude"]).float()[:, None, :]
    sin = (torch.sin(angle) * (sign * s["magnitude"])).float()[:, None, :]
    h, rot = c["rot"] // 2, c["rot"]

    def turn(x):
        y = x.float()
        if c["layout"] == "half":
            a, b = y[..., :h], y[..., h:rot]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        return torch.cat([r, y[..., rot:]], dim=-1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _act(name, x):
    return x if name == "none" else torch.sigmoid(x) * (x if name == "silu" else 1.0)


EPS = 1e-5


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if c["gate"] == "before":
        x = x * _act(c["act"], s["z"].float())
    if c["kind"] == "mean":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    y = y if s["w"] is None else y * s["w"]
    y = y if s["b"] is None else y + s["b"]
    if c["gate"] == "after":
        y = y * _act(c["act"], s["z"].float())
    elif c["gate"] == "none":
        y = _act(c["act"], y)
    return y.to(DT[c["out"]])


# ---------------------------------------------------------------------------
# The package's entry points
# ---------------------------------------------------------------------------

def _handle(s, lq):
    """What a program makes once for a layer and keeps: the configuration, and
    the prompt's workspace or the rotary table."""
    c = s["case"]
    if c["op"] in ("prompt", "token"):
        cfg = lq.make_linear_config(
            c["seqs"], c["hk"], c["hv"], c["dk"], c["dv"],
            decay=lq.LQ_DECAY_TOKEN if c["decay"] == "token" else lq.LQ_DECAY_HEAD, in_bf16=c["io"] == BF16,
            out_bf16=c["out"] == BF16, q_stride=s["q"].stride(0), k_stride=s["k"].stride(0),
            v_stride=s["v"].stride(0))
        space = lq.lq_linear_workspace_bytes(cfg, c["tokens"]) if c["op"] == "prompt" else 0
        return cfg, torch.empty(max(space, 16), dtype=torch.uint8, device="cuda")
    if c["op"] == "rotary":
        kind = {"none": lq.LQ_ROPE_NONE, "linear": lq.LQ_ROPE_LINEAR, "ntk": lq.LQ_ROPE_NTK,
                "parts": lq.LQ_ROPE_PARTS}[c["scaling"]]
        table, magnitude = lq.lq_rotary_table(c["rot"], THETA, kind, factor=FACTOR, trained=TRAINED,
                                              fast_turns=FAST, slow_turns=SLOW)
        cfg = lq.make_rotary_config(
            c["hq"], c["hk"], c["d"], c["rot"],
            layout=lq.LQ_ROPE_HALF if c["layout"] == "half" else lq.LQ_ROPE_INTERLEAVED, bf16=c["io"] == BF16,
            magnitude=magnitude, inverse=c["inverse"], q_stride=s["q"].stride(0), k_stride=s["k"].stride(0))
        return cfg, table.cuda()
    cfg = lq.make_norm_config(
        c["groups"], c["size"], kind=lq.LQ_NORM_RMS if c["kind"] == "rms" else lq.LQ_NORM_MEAN,
        act={"none": lq.LQ_ACT_NONE, "silu": lq.LQ_ACT_SILU, "sigmoid": lq.LQ_ACT_SIGMOID}[c["act"]],
        gate_before=c["gate"] == "before", shared_weight=c["weight"] == "group", in_bf16=c["io"] == BF16,
        out_bf16=c["out"] == BF16, eps=EPS)
    return cfg, None


def _own_run(s):
    from recurrent_state_quantization_decode_b200 import binding as lq

    if "handle" not in s:
        s["handle"] = _handle(s, lq)
    cfg, extra = s["handle"]
    op = s["case"]["op"]
    if op == "prompt":
        lq.lq_linear_prefill(cfg, s["q"], s["k"], s["v"], s["decay"], s["case"]["tokens"], s["offsets"], s["S"],
                             s["S"].shape[0], s["out"], s["err"], slots=s["slots"], fresh=s["fresh"],
                             workspace=extra)
        return s["out"], s["S"]
    if op == "token":
        lq.lq_linear_decode_step(cfg, s["q"], s["k"], s["v"], s["decay"], s["S"], s["S"].shape[0], s["out"],
                                 s["err"], slots=s["slots"])
        return s["out"], s["S"]
    if op == "rotary":
        lq.lq_rotary(cfg, s["case"]["tokens"], s["q"], s["k"], s["positions"], extra, s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    lq.lq_group_norm(cfg, s["case"]["tokens"], s["x"], s["out"], gate=s["z"], weight=s["w"], bias=s["b"])
    return s["out"]


PLAIN = {"prompt": _plain_prompt, "token": _plain_token, "rotary": _plain_rotary, "norm": _plain_norm}


def run(state):
    if own:
        return _own_run(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c, size = case, {BF16: 2, F32: 4}
    if c["op"] in ("prompt", "token"):
        n = c["tokens"] if c["op"] == "prompt" else c["seqs"]
        tile = c["hv"] * c["dv"] * c["dk"]
        reads = c["seqs"]  # sequences whose first state is read
        if c["op"] == "prompt":
            reads = 0 if c["fresh"] else c["seqs"] - -(-c["seqs"] // 3)
        io = n * (2 * c["hk"] * c["dk"] + c["hv"] * c["dv"]) * size[c["io"]] + n * c["hv"] * c["dv"] * size[c["out"]]
        gates = 4 * c["hv"] * (n if c["decay"] == "token" else 1)
        # the recurrence itself: a decayed rank-1 update and a product with q per token
        return {"bytes": io + gates + 4 * tile * (c["seqs"] + reads), "flops": 5 * n * tile}
    if c["op"] == "rotary":
        x = c["tokens"] * (c["hq"] + c["hk"])
        return {"bytes": 2 * x * c["d"] * size[c["io"]] + 4 * c["tokens"] + 4 * c["rot"], "flops": 3 * x * c["rot"]}
    x = c["tokens"] * c["groups"] * c["size"]
    params = ({"none": 0, "group": c["size"], "channel": c["groups"] * c["size"]}[c["weight"]]
              + (c["groups"] * c["size"] if c["bias"] else 0))
    ins = 1 if c["gate"] == "none" else 2
    return {"bytes": x * (ins * size[c["io"]] + size[c["out"]]) + 4 * params, "flops": 6 * x}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_recurrence(s, case, off):
    """Token by token: S <- a S + v k^T, o = S q, all sequences side by side."""
    n, hk, hv, dk, dv = case["seqs"], case["hk"], case["hv"], case["dk"], case["dv"]
    lengths = [off[b + 1] - off[b] for b in range(n)]
    slot = s["slots"].long()
    states = s["S"].double()
    S = states[slot]
    if "fresh" in s:
        S[s["fresh"].bool()] = 0.0
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    out = torch.zeros((off[-1], hv, dv), dtype=torch.float64, device="cuda")
    order = sorted(range(n), key=lambda b: -lengths[b])  # the longest first: the running ones are a prefix
    S = S[order].reshape(n, hk, hv // hk, dv, dk)
    starts = torch.tensor([off[b] for b in order], device="cuda")
    live = n
    for t in range(max(lengths)):
        while lengths[order[live - 1]] <= t:
            live -= 1
        at = starts[:live] + t
        a = s["decay"][at] if case["decay"] == "token" else s["decay"].expand(live, hv)
        part = S[:live]
        part.mul_(a.double().reshape(live, hk, -1, 1, 1))
        part.addcmul_(v[at].reshape(live, hk, -1, dv, 1), k[at][:, :, None, None, :])
        o = torch.matmul(part, q[at][:, :, None, :, None])
        out[at] = o.reshape(live, hv, dv)
    states[slot[order]] = S.reshape(n, hv, dv, dk)
    return out, states


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_recurrence(s, case, s["offsets"].tolist())
    if case["op"] == "token":
        return _exact_recurrence(s, case, list(range(case["seqs"] + 1)))
    if case["op"] == "rotary":
        # a rotation is a product of complex numbers
        turn = torch.polar(torch.full((case["rot"] // 2,), s["magnitude"], dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None] * s["freq"])[:, None, :]
        turn = turn.conj() if case["inverse"] else turn

        def of(x):
            y, r = x.double(), case["rot"]
            half = case["layout"] == "half"
            pairs = y[..., :r].unflatten(-1, (2, r // 2) if half else (r // 2, 2))
            pairs = pairs.transpose(-1, -2) if half else pairs
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.transpose(-1, -2) if half else z
            return torch.cat([z.flatten(-2), y[..., r:]], dim=-1)

        return of(s["q"]), of(s["k"])
    x, z = s["x"].double(), None if s["z"] is None else s["z"].double()
    act = {"none": lambda t: t, "silu": lambda t: t / (1 + torch.exp(-t)),
           "sigmoid": lambda t: 1 / (1 + torch.exp(-t))}[case["act"]]
    if case["gate"] == "before":
        x = x * act(z)
    mean = x.mean(-1, keepdim=True) if case["kind"] == "mean" else torch.zeros_like(x[..., :1])
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS)
    y = y * (1.0 if s["w"] is None else s["w"].double()) + (0.0 if s["b"] is None else s["b"].double())
    return y * act(z) if case["gate"] == "after" else act(y) if case["gate"] == "none" else y
