"""The layer operators on the GPU against their definitions in 64 bits.

Bounds.  u = 2^-24 is half a step of fp32, r = 2^-8 of bf16.  Write A for an
output computed with absolute values everywhere (|a|, |k|, |q|, |v|, |S|).
  * One token: S' = a S + v k rounds the product and the sum (2 u of the
    absolute state); o sums dk products of it (dk u A more): u (dk + 4) A.
  * A prompt: a term passes at most 2 roundings a token on its way through the
    state and dk + 2 in the dot product: u (2 T + dk + 4) A from the token form.
    The chunked form adds at most, a term: the exponential of its decay (a few
    u), three-part splits of its operands (u each), sums of up to 128 + dk terms
    in the chunk, and one sum a chunk: within the same bound, T being rounded up
    to a whole chunk of 128.  With bf16 outputs it may round the scores and the
    state once to bf16 before a product: 2 r A more.
  * bf16 outputs: r |o| for the final rounding.
These are worst cases; random roundings stay far below them, so outputs and
states are also held to a relative 2-norm error of 1e-5 (fp32 results) and
2 r (bf16 results: up to three roundings of r / sqrt(3) in quadrature).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U, R = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def B():
    from recurrent_state_quantization_decode_b200 import binding

    return binding


def _unit(x):
    return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True).clamp_min(1e-6)


class Linear:
    """Seeded inputs of packed sequences and the recurrence in 64 bits."""

    def __init__(self, lengths, hk, hv, dk, dv, io=BF, out=BF, decay="token", fused=False, seed=0, spare=2,
                 tail=0, alpha=None):
        self.lengths, self.hk, self.hv, self.dk, self.dv = list(lengths), hk, hv, dk, dv
        self.io, self.out_dtype, self.decay_kind = io, out, decay
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = sum(lengths)
        self.n, self.rows, self.b = n, n + tail, len(lengths)

        def rnd(*s):
            return torch.randn(s, generator=g, device="cuda")

        q, k, v = _unit(rnd(self.rows, hk, dk)), _unit(rnd(self.rows, hk, dk)), rnd(self.rows, hv, dv)
        q[n:], k[n:], v[n:] = math.nan, math.inf, math.nan  # rows behind the last sequence: never read as tokens
        q, k, v = q.to(io), k.to(io), v.to(io)
        if fused:
            rows = torch.cat([x.reshape(self.rows, -1) for x in (q, k, v)], dim=1)
            a, c = hk * dk, hv * dv
            q = rows[:, :a].unflatten(1, (hk, dk))
            k = rows[:, a:2 * a].unflatten(1, (hk, dk))
            v = rows[:, 2 * a:2 * a + c].unflatten(1, (hv, dv))
        self.q, self.k, self.v = q, k, v
        if decay == "head":
            self.decay = torch.exp(-torch.exp2(-8.0 * torch.arange(1, hv + 1, device="cuda") / hv))
        else:
            self.decay = 0.9 + 0.1 * torch.rand((self.rows, hv), generator=g, device="cuda")
        if alpha is not None:
            self.decay = alpha(self.decay, g)
        self.num_slots = self.b + spare
        self.S = 0.1 * rnd(self.num_slots, hv, dv, dk)
        self.slots = torch.randperm(self.num_slots, generator=torch.Generator().manual_seed(seed))[:self.b]
        self.slots = self.slots.to(torch.int32).cuda()
        off = [0]
        for x in lengths:
            off.append(off[-1] + x)
        self.off = off
        self.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        self.fresh = None
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def cfg(self, B, **kw):
        return B.make_linear_config(
            self.b, self.hk, self.hv, self.dk, self.dv,
            decay=B.LQ_DECAY_HEAD if self.decay_kind == "head" else B.LQ_DECAY_TOKEN, in_bf16=self.io == BF,
            out_bf16=self.out_dtype == BF, q_stride=self.q.stride(0), k_stride=self.k.stride(0),
            v_stride=self.v.stride(0), **kw)

    def new_out(self):
        return torch.full((self.rows, self.hv, self.dv), 7.0, dtype=self.out_dtype, device="cuda")

    def workspace(self, B, cfg):
        return torch.empty(max(16, B.lq_linear_workspace_bytes(cfg, self.n)), dtype=torch.uint8, device="cuda")

    def prefill(self, B, S, out, ws=None, cfg=None, **kw):
        cfg = cfg or self.cfg(B)
        ws = self.workspace(B, cfg) if ws is None else ws
        B.lq_linear_prefill(cfg, self.q, self.k, self.v, self.decay, self.n, self.offsets, S, self.num_slots, out,
                            self.err, slots=self.slots, fresh=self.fresh, workspace=ws, **kw)
        return ws

    def exact(self, absolute=False, skip=()):
        """(out, pool) in 64 bits; with `absolute`, of the absolute values."""
        mag = (lambda x: x.double().abs()) if absolute else (lambda x: x.double())
        q, k, v, d = mag(self.q[:self.n]), mag(self.k[:self.n]), mag(self.v[:self.n]), mag(self.decay)
        pool, rep = mag(self.S).clone(), self.hv // self.hk
        out = torch.zeros((self.n, self.hv, self.dv), dtype=torch.float64, device="cuda")
        for b in range(self.b):
            if b in skip:
                continue
            S = pool[int(self.slots[b])].clone()
            if self.fresh is not None and int(self.fresh[b]):
                S.zero_()
            for t in range(self.off[b], self.off[b + 1]):
                a = d if self.decay_kind == "head" else d[t]
                S = a[:, None, None] * S + v[t][:, :, None] * k[t].repeat_interleave(rep, 0)[:, None, :]
                out[t] = torch.einsum("hvk,hk->hv", S, q[t].repeat_interleave(rep, 0))
            pool[int(self.slots[b])] = S
        return out, pool

    def check(self, out, S, skip=()):
        """out and S against the bounds above; other slots and rows untouched."""
        assert int(self.err) == 0
        eo, es = self.exact(skip=skip)
        ao, as_ = self.exact(absolute=True, skip=skip)
        T = -(-max(self.lengths) // 128) * 128
        c = U * (2 * T + self.dk + 4)
        used = [int(self.slots[b]) for b in range(self.b) if b not in skip]
        idle = [i for i in range(self.num_slots) if i not in used]
        assert torch.equal(S[idle], self.S[idle])
        ds = (S.double() - es).abs()
        assert bool((ds <= c * as_ + 1e-30).all()), float((ds / (as_ + 1e-30)).max())
        assert float(torch.linalg.vector_norm(ds)) <= 1e-5 * float(torch.linalg.vector_norm(es)) + 1e-30
        if out is None:
            return
        assert bool((out[self.n:] == 7.0).all())
        live = torch.ones(self.n, dtype=torch.bool, device="cuda")
        for b in skip:
            live[self.off[b]:self.off[b + 1]] = False
            assert bool((out[self.off[b]:self.off[b + 1]] == 7.0).all())
        o, eo, ao = out[:self.n][live].double(), eo[live], ao[live]
        bf = self.out_dtype == BF
        do = (o - eo).abs()
        lim = (c + (2 * R if bf else 0.0)) * ao + (R if bf else U) * eo.abs() + 1e-30
        assert bool((do <= lim).all()), float((do / lim).max())
        rel = 2 * R if bf else 1e-5
        assert float(torch.linalg.vector_norm(do)) <= rel * float(torch.linalg.vector_norm(eo)) + 1e-30


# ---------------------------------------------------------------------------
# Linear attention: one token
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("io,out", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_step_matches_the_definition(B, dk, dv, io, out):
    c = Linear([1] * 5, 3, 6, dk, dv, io, out, fused=dk == 64, seed=dk + dv)
    S, o = c.S.clone(), c.new_out()
    B.lq_linear_decode_step(c.cfg(B), c.q, c.k, c.v, c.decay, S, c.num_slots, o, c.err, slots=c.slots)
    c.check(o, S)


@pytest.mark.parametrize("batch,hk,hv,decay", [(1, 1, 1, "head"), (1, 16, 32, "token"), (67, 2, 2, "head"),
                                               (300, 1, 4, "token")])
def test_step_batches(B, batch, hk, hv, decay):
    c = Linear([1] * batch, hk, hv, 128, 128, BF, F32, decay=decay, seed=batch)
    S, o = c.S.clone(), c.new_out()
    B.lq_linear_decode_step(c.cfg(B), c.q, c.k, c.v, c.decay, S, c.num_slots, o, c.err, slots=c.slots)
    c.check(o, S)


def test_step_without_slots_uses_the_sequence_number(B):
    c = Linear([1] * 3, 1, 2, 64, 64, F32, F32, spare=0)
    c.slots = torch.arange(3, dtype=torch.int32, device="cuda")
    S, o = c.S.clone(), c.new_out()
    B.lq_linear_decode_step(c.cfg(B), c.q, c.k, c.v, c.decay, S, c.num_slots, o, c.err)
    c.check(o, S)


def _bad_slots(B, c, call):
    """Negative slots skip; a slot past the pool and one named twice are skipped and reported."""
    own = c.slots.clone()
    # (slots, sequences left out, whether it is reported)
    for change, skip, report in (({1: -1}, {1}, False), ({2: -7}, {2}, False), ({0: c.num_slots}, {0}, True),
                                 ({3: 1 << 30}, {3}, True), ({3: int(own[1])}, {3}, True),
                                 ({0: -1, 2: -1}, {0, 2}, False), ({4: int(own[0]), 3: int(own[0])}, {3, 4}, True)):
        c.slots = own.clone()
        for i, s in change.items():
            c.slots[i] = s
        S, o = c.S.clone(), c.new_out()
        call(S, o)
        assert B.lq_get_error_word(c.err) == (B.LQ_ERR_DEVICE_BOUNDS if report else B.LQ_OK), change
        assert B.lq_get_error_word(c.err) == B.LQ_OK
        c.check(o, S, skip=skip)


def test_step_slots_that_cannot_be_used(B):
    c = Linear([1] * 5, 2, 4, 64, 128, BF, F32)
    _bad_slots(B, c, lambda S, o: B.lq_linear_decode_step(c.cfg(B), c.q, c.k, c.v, c.decay, S, c.num_slots, o,
                                                          c.err, slots=c.slots))


# ---------------------------------------------------------------------------
# Linear attention: prompts
# ---------------------------------------------------------------------------

RAGGED = [0, 1, 5, 127, 128, 129, 0, 255, 300, 16, 513]

PROMPTS = {
    "bf16_d128_ragged": dict(lengths=RAGGED, hk=2, hv=4, dk=128, dv=128),
    "bf16_d128_fused_f32_out": dict(lengths=RAGGED, hk=2, hv=2, dk=128, dv=128, out=F32, fused=True),
    "bf16_d64_ragged": dict(lengths=RAGGED, hk=1, hv=4, dk=64, dv=64, fused=True),
    "bf16_d64_f32_out": dict(lengths=[129, 64, 3], hk=3, hv=3, dk=64, dv=64, out=F32),
    "bf16_d32": dict(lengths=RAGGED, hk=2, hv=2, dk=32, dv=32, out=F32),
    "bf16_k128_v64": dict(lengths=[70, 0, 401], hk=1, hv=2, dk=128, dv=64),
    "bf16_k64_v128": dict(lengths=[70, 0, 401], hk=1, hv=2, dk=64, dv=128, out=F32),
    "bf16_k32_v128": dict(lengths=[200], hk=1, hv=3, dk=32, dv=128),
    "bf16_k128_v32": dict(lengths=[1, 200], hk=5, hv=5, dk=128, dv=32),
    "bf16_one_token": dict(lengths=[1], hk=4, hv=8, dk=128, dv=128),
    "bf16_head_decay": dict(lengths=[700, 90], hk=4, hv=8, dk=128, dv=128, decay="head", out=F32),
    "bf16_many": dict(lengths=[37 * i % 400 for i in range(60)], hk=4, hv=8, dk=128, dv=128),
    "bf16_many_f32_out": dict(lengths=[53 * i % 300 for i in range(150)], hk=1, hv=3, dk=64, dv=128, out=F32),
    "f32_many": dict(lengths=[29 * i % 200 for i in range(140)], hk=1, hv=2, dk=32, dv=64, io=F32, out=F32),
    "bf16_long": dict(lengths=[3001], hk=2, hv=2, dk=128, dv=128, decay="head"),
    "bf16_long_f32_out": dict(lengths=[40, 2500], hk=1, hv=1, dk=128, dv=128, out=F32),
    "f32_d128_ragged": dict(lengths=RAGGED, hk=2, hv=4, dk=128, dv=128, io=F32, out=F32),
    "f32_d64_bf16_out": dict(lengths=RAGGED, hk=1, hv=2, dk=64, dv=64, io=F32, out=BF, fused=True),
    "f32_d32": dict(lengths=[33, 1, 31], hk=2, hv=2, dk=32, dv=32, io=F32, out=F32, decay="head"),
    "f32_k32_v128": dict(lengths=[300, 20], hk=1, hv=2, dk=32, dv=128, io=F32, out=F32),
    "f32_long": dict(lengths=[2100], hk=1, hv=2, dk=64, dv=128, io=F32, out=F32, decay="head"),
}


@pytest.mark.parametrize("name", sorted(PROMPTS))
@pytest.mark.parametrize("fresh", ["none", "some"])
def test_prefill_matches_the_definition(B, name, fresh):
    c = Linear(**PROMPTS[name], seed=len(name), tail=9)
    if fresh == "some":
        c.fresh = (torch.arange(c.b) % 2 == 0).to(torch.int32).cuda()
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o)
    c.check(o, S)
    # the same call on the same inputs gives the same bits
    S2, o2 = c.S.clone(), c.new_out()
    c.prefill(B, S2, o2)
    assert torch.equal(S, S2) and torch.equal(o, o2)
    # states alone
    S3 = c.S.clone()
    c.prefill(B, S3, None)
    c.check(None, S3)


def _zeros(d, g):
    d = d.clone()
    d[torch.rand(d.shape, generator=g, device="cuda") < 0.05] = 0.0
    return d


DECAYS = {
    "zeros": _zeros,                                            # resets inside chunks and between them
    "all_zero": lambda d, g: torch.zeros_like(d),
    "ones": lambda d, g: torch.ones_like(d),
    "tiny": lambda d, g: torch.full_like(d, 1e-30),             # a product of two underflows
    "small": lambda d, g: 0.3 * torch.rand(d.shape, generator=g, device="cuda"),
    "denormal": lambda d, g: torch.where(torch.rand(d.shape, generator=g, device="cuda") < 0.5, 1e-41, 0.99),
    "close_to_one": lambda d, g: 1.0 - 1e-3 * torch.rand(d.shape, generator=g, device="cuda"),
}


@pytest.mark.parametrize("kind", sorted(DECAYS))
@pytest.mark.parametrize("io,out", [(BF, BF), (BF, F32), (F32, F32)])
def test_prefill_decays(B, kind, io, out):
    c = Linear([300, 64, 511], 1, 2, 128, 128, io, out, seed=3, alpha=DECAYS[kind])
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o)
    c.check(o, S)


def test_prefill_slots_that_cannot_be_used(B):
    for io in (BF, F32):
        c = Linear([150, 3, 40, 129, 70], 2, 4, 128, 64, io, F32)
        _bad_slots(B, c, lambda S, o: c.prefill(B, S, o))


@pytest.mark.parametrize("io", [BF, F32])
def test_prefill_offsets_that_are_not_ascending(B, io):
    """A sequence whose offsets leave the rows or run backwards is left out and reported."""
    c = Linear([20, 150, 30], 1, 2, 128, 128, io, F32)
    for bad in ([-1, 150, 180, 200], [0, 150, 100, 200], [0, 20, 170, 201], [0, 20, 1 << 30, 200]):
        c.offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
        S, o = c.S.clone(), c.new_out()
        c.prefill(B, S, o)
        assert B.lq_get_error_word(c.err) == B.LQ_ERR_DEVICE_BOUNDS
        for b in range(3):
            if not 0 <= bad[b] <= bad[b + 1] <= c.n:
                assert torch.equal(S[int(c.slots[b])], c.S[int(c.slots[b])])


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("pairs", [3, 40, 90])
def test_prefill_offsets_that_start_over(B, io, pairs):
    """Offsets that go back are a fault from there on: the sequences before are computed, and the
    workspace, which could not hold overlapping sequences, is not left."""
    n = 64 * pairs + 508  # more than 32 a sequence: bf16 takes the chunks
    c = Linear([n] + [0] * (2 * pairs - 2), 1, 2, 128, 128, io, F32)
    c.offsets = torch.tensor(([0, n] * pairs)[:2 * pairs], dtype=torch.int32, device="cuda")
    size = B.lq_linear_workspace_bytes(c.cfg(B), n)
    ws = torch.full((size + (64 << 20),), 171, dtype=torch.uint8, device="cuda")
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o, ws=ws[:size] if size else None)
    assert bool((ws[size:] == 171).all())
    assert B.lq_get_error_word(c.err) == B.LQ_ERR_DEVICE_BOUNDS
    c.err.zero_()
    c.check(o, S, skip=range(1, c.b))
    # offsets that leave the rows but ascend: only the sequences past the rows are left out
    d = Linear([n, 0, 5], 1, 2, 128, 128, io, F32)
    d.offsets = torch.tensor([0, n, n + 9, n + 9], dtype=torch.int32, device="cuda")
    S, o = d.S.clone(), d.new_out()
    d.prefill(B, S, o)
    assert B.lq_get_error_word(d.err) == B.LQ_ERR_DEVICE_BOUNDS
    d.err.zero_()
    d.check(o, S, skip=(1, 2))


@pytest.mark.parametrize("io,out", [(BF, BF), (BF, F32), (F32, F32)])
def test_prefill_values_that_are_not_finite(B, io, out):
    """They stay in their sequence, head and channel, and in bf16 prompts within their chunk before
    their token (fp32 prompts: not before it at all)."""
    c = Linear([300, 150], 1, 2, 128, 128, io, out, seed=8)
    S0, o0 = c.S.clone(), c.new_out()
    c.prefill(B, S0, o0)
    for bad in (math.inf, math.nan):
        v = c.v.clone()
        c.v[200, 1, 37] = bad
        S, o = c.S.clone(), c.new_out()
        c.prefill(B, S, o)
        c.v = v
        assert not bool(o[200:300, 1, 37].isfinite().any())
        assert not bool(S[int(c.slots[0]), 1, 37].isfinite().any())
        o[200:300, 1, 37] = o0[200:300, 1, 37]
        if io == BF:
            o[128:200, 1, 37] = o0[128:200, 1, 37]
        S[int(c.slots[0]), 1, 37] = S0[int(c.slots[0]), 1, 37]
        assert torch.equal(o, o0) and torch.equal(S, S0)
    assert int(c.err) == 0


def test_prefill_then_steps_is_one_prefill(B):
    """A prompt in two calls and single tokens end where one call ends."""
    for io, out in ((BF, F32), (F32, F32)):
        c = Linear([200, 333], 2, 4, 128, 128, io, out, seed=11, spare=0)
        c.slots = torch.arange(2, dtype=torch.int32, device="cuda")
        S, o = c.S.clone(), c.new_out()
        cut = [150, 300]
        rows = [torch.arange(c.off[b], c.off[b] + cut[b], device="cuda") for b in range(2)]
        at = torch.cat(rows)
        off = torch.tensor([0, cut[0], sum(cut)], dtype=torch.int32, device="cuda")
        cfg = B.make_linear_config(2, 2, 4, 128, 128, in_bf16=io == BF)
        ws = torch.empty(max(16, B.lq_linear_workspace_bytes(cfg, sum(cut))), dtype=torch.uint8, device="cuda")
        part = torch.empty((sum(cut), 4, 128), device="cuda")
        B.lq_linear_prefill(cfg, c.q[at], c.k[at], c.v[at], c.decay[at], sum(cut), off, S, 2, part, c.err,
                            workspace=ws)
        o[at] = part
        one = torch.empty((2, 4, 128), device="cuda")
        for t in range(50):  # sequence 0 ends after 50 more tokens, sequence 1 after 33
            live = [b for b in range(2) if cut[b] + t < c.lengths[b]]
            tok = torch.tensor([c.off[b] + min(cut[b] + t, c.lengths[b] - 1) for b in range(2)], device="cuda")
            slots = torch.tensor([b if b in live else -1 for b in range(2)], dtype=torch.int32, device="cuda")
            B.lq_linear_decode_step(cfg, c.q[tok], c.k[tok], c.v[tok], c.decay[tok], S, 2, one, c.err, slots=slots)
            for b in live:
                o[c.off[b] + cut[b] + t] = one[b]
        c.check(o, S)


def test_prefill_captured_and_on_another_stream(B):
    c = Linear([260, 40], 2, 2, 128, 128, BF, BF, seed=5)
    S0, o0 = c.S.clone(), c.new_out()
    c.prefill(B, S0, o0)
    # two calls at once, each with a workspace of its own
    S1, o1, S2, o2 = c.S.clone(), c.new_out(), c.S.clone(), c.new_out()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = c.workspace(B, c.cfg(B)), c.workspace(B, c.cfg(B))
    torch.cuda.synchronize()
    c.prefill(B, S1, o1, ws=w1, stream=a)
    c.prefill(B, S2, o2, ws=w2, stream=b)
    torch.cuda.synchronize()
    for S, o in ((S1, o1), (S2, o2)):
        assert torch.equal(S, S0) and torch.equal(o, o0)
    # captured, then replayed on new contents of the same buffers
    S3, o3, w3 = c.S.clone(), c.new_out(), c.workspace(B, c.cfg(B))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.prefill(B, S3, o3, ws=w3)
    for _ in range(2):
        S3.copy_(c.S)
        o3.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(S3, S0) and torch.equal(o3, o0)
    assert int(c.err) == 0


def test_states_past_32_bit_offsets(B):
    """A slot whose state starts more than 2^31 values into the pool."""
    c = Linear([2], 32, 32, 128, 128, BF, F32, spare=0)
    slots = (1 << 31) // (32 * 128 * 128) + 3
    pool = torch.empty((slots, 32, 128, 128), device="cuda")
    small = c.S.clone()
    pool[slots - 1] = small[0]
    o, big = c.new_out(), torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    B.lq_linear_prefill(c.cfg(B), c.q, c.k, c.v, c.decay, 2, c.offsets, pool, slots, o, c.err, slots=big,
                        workspace=c.workspace(B, c.cfg(B)))
    c.slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(o, pool[slots - 1:].clone())
    step = Linear([1], 32, 32, 128, 128, BF, F32, spare=0)
    pool[slots - 1] = step.S[0]
    o = step.new_out()
    B.lq_linear_decode_step(step.cfg(B), step.q, step.k, step.v, step.decay, pool, slots, o, step.err, slots=big)
    step.slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    step.check(o, pool[slots - 1:].clone())


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

def _rotated(x, pos, freq, mag, layout, rot, inverse):
    """(exact, bound) in 64 bits.  The angle in turns is exact to 2^-33, fp32
    rounding of it and of sin and cos to 2 steps: 4 u each of |a| + |b|; products
    and sum 2 u more, and the magnitude's 2; then the output's rounding."""
    y = x.double()
    ang = pos.double()[:, None] * freq
    co, si = (torch.cos(ang) * mag)[:, None], (torch.sin(ang) * mag * (-1 if inverse else 1))[:, None]
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if layout == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    na, nb = a * co - b * si, b * co + a * si
    size = (a.abs() + b.abs()) * mag
    join = (lambda u, v: torch.cat([u, v], -1)) if layout == "half" else \
        (lambda u, v: torch.stack([u, v], -1).flatten(-2))
    out = torch.cat([join(na, nb), y[..., rot:]], -1)
    bound = torch.cat([join(size, size) * 16 * U, torch.zeros_like(y[..., rot:])], -1)
    half_step = R if x.dtype == BF else U
    return out, bound + half_step * out.abs() * (1 + R)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("n,hq,hk,d,rot", [(1, 1, 1, 128, 128), (7, 5, 2, 128, 64), (3, 2, 1, 80, 78),
                                           (33, 3, 3, 64, 14), (2000, 4, 1, 128, 96), (5, 0, 2, 32, 32),
                                           (9, 7, 0, 256, 256), (4, 1, 2, 2, 2), (6, 2, 2, 1024, 1024),
                                           (5, 3, 1, 77, 40)])
def test_rotary_matches_the_definition(B, layout, io, n, hq, hk, d, rot):
    g = torch.Generator(device="cuda").manual_seed(n + d)
    rows = torch.randn((n, (hq + hk) * d), generator=g, device="cuda").to(io)
    q = rows[:, :hq * d].unflatten(1, (hq, d)) if hq else None
    k = rows[:, hq * d:].unflatten(1, (hk, d)) if hk else None
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (n,), generator=g, device="cuda").to(torch.int32)
    pos[0] = (1 << 31) - 1
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    table, _ = B.lq_rotary_table(rot)
    table = table.cuda()
    lay = B.LQ_ROPE_HALF if layout == "half" else B.LQ_ROPE_INTERLEAVED
    for inverse, mag in ((False, 1.0), (True, 1.25)):
        def cfg(**kw):
            return B.make_rotary_config(hq, hk, d, rot, layout=lay, bf16=io == BF, magnitude=mag, inverse=inverse,
                                        q_stride=rows.stride(0) if hq else 0, k_stride=rows.stride(0) if hk else 0,
                                        **kw)

        qo = torch.empty((n, hq, d), dtype=io, device="cuda") if hq else None
        ko = torch.empty((n, hk, d), dtype=io, device="cuda") if hk else None
        B.lq_rotary(cfg(), n, q, k, pos, table, qo, ko)
        # 2^31 f in 64-bit floating point is off by 2^-22 of a radian at most, the table by as little
        for x, y in ((q, qo), (k, ko)):
            if x is None:
                continue
            want, bound = _rotated(x, pos, freq, mag, layout, rot, inverse)
            slack = 2.0 ** -20 * mag * x.double().abs().amax()
            assert bool(((y.double() - want).abs() <= bound + slack).all())
            assert torch.equal(y[..., rot:], x[..., rot:])
        # in place, on the fused rows
        own = rows.clone()
        iq = own[:, :hq * d].unflatten(1, (hq, d)) if hq else None
        ik = own[:, hq * d:].unflatten(1, (hk, d)) if hk else None
        B.lq_rotary(cfg(q_out_stride=rows.stride(0) if hq else 0, k_out_stride=rows.stride(0) if hk else 0), n, iq,
                    ik, pos, table, iq, ik)
        for x, y in ((iq, qo), (ik, ko)):
            assert x is None or torch.equal(x, y)


def test_rotary_near_positions_are_tight(B):
    """Within 2^20 positions the 64-bit reference itself is exact to 2^-33: the bound alone."""
    for layout in ("half", "interleaved"):
        g = torch.Generator(device="cuda").manual_seed(1)
        q = torch.randn((500, 2, 64), generator=g, device="cuda")
        pos = torch.randint(0, 1 << 20, (500,), generator=g, device="cuda", dtype=torch.int32)
        pos[:3] = torch.tensor([0, 1, 2])
        freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device="cuda") / 64)
        table, _ = B.lq_rotary_table(64)
        out = torch.empty_like(q)
        cfg = B.make_rotary_config(2, 0, 64, 64, bf16=False,
                                   layout=B.LQ_ROPE_HALF if layout == "half" else B.LQ_ROPE_INTERLEAVED)
        B.lq_rotary(cfg, 500, q, None, pos, table.cuda(), out, None)
        want, bound = _rotated(q, pos, freq, 1.0, layout, 64, False)
        assert bool(((out.double() - want).abs() <= bound).all())
        assert torch.equal(out[0], q[0])  # position 0 turns nothing


# ---------------------------------------------------------------------------
# Group norm
# ---------------------------------------------------------------------------

def _act(B, kind, x):
    return x if kind == B.LQ_ACT_NONE else torch.sigmoid(x) * (x if kind == B.LQ_ACT_SILU else 1.0)


def _check_norm(B, n, groups, size, kind, act, gate, before, shared, weight, bias, io, out, seed=0, misalign=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda")

    row, pad = groups * size, (3 if misalign else 0)
    x = (rnd(n, row + pad) * 2 + 0.5).to(io)[:, pad:].unflatten(1, (groups, size))
    z = rnd(n, row + pad).to(io)[:, pad:].unflatten(1, (groups, size)) if gate else None
    w = (1 + 0.3 * rnd(*((size,) if shared else (groups, size)))) if weight else None
    b = 0.2 * rnd(groups, size) if bias else None
    y = torch.full((n + 1, groups, size), 7.0, dtype=out, device="cuda")
    cfg = B.make_norm_config(groups, size, kind=kind, act=act, gate_before=before, shared_weight=shared,
                             in_bf16=io == BF, out_bf16=out == BF, eps=1e-5, x_stride=row + pad,
                             gate_stride=row + pad if gate else 0)
    B.lq_group_norm(cfg, n, x, y[:n], gate=z, weight=w, bias=b)
    assert bool((y[n] == 7.0).all())
    xd, zd = x.double(), None if z is None else z.double()
    if before:
        xd = xd * _act(B, act, zd)
    mean = xd.mean(-1, keepdim=True) if kind == B.LQ_NORM_MEAN else 0.0
    c = xd - mean
    s = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    wd = 1.0 if w is None else w.double()
    nx = c * s * wd + (0.0 if b is None else b.double())
    want = nx * _act(B, act, zd) if gate and not before else nx if gate else _act(B, act, nx)
    # sums of `size` terms: (size + 4) u of the mean's absolute terms on c, the same relative on s; an
    # activation is Lipschitz with 1.1 and computed to 8 u relative of itself (|x| u in its exponent)
    e = (size + 12) * U
    mag = (xd.abs() + (xd.abs().mean(-1, keepdim=True) if kind == B.LQ_NORM_MEAN else 0.0)) * s
    spread = (mag * (wd.abs() if weight else 1.0) + nx.abs()) * e * 3
    if gate and not before:
        lim = spread * _act(B, act, zd).abs() + want.abs() * (12 + zd.abs()) * U
    elif gate or act == B.LQ_ACT_NONE:
        lim = spread
    else:
        lim = 1.1 * spread + want.abs() * (12 + nx.abs()) * U
    if before:  # the gate's own error, through the norm
        lim = lim + (12 + zd.abs().amax()) * U * mag * 2 * (wd.abs().amax() if weight else 1.0)
    lim = lim * (1 + R) + (R if out == BF else U) * want.abs() + 1e-30
    d = (y[:n].double() - want).abs()
    assert bool((d <= lim).all()), float((d / lim).max())
    rel = R if out == BF else 2e-6
    assert float(torch.linalg.vector_norm(d)) <= rel * float(torch.linalg.vector_norm(want))


@pytest.mark.parametrize("size", [1, 2, 7, 16, 32, 64, 100, 128, 129, 333, 512, 1024, 1500, 4096, 8192])
@pytest.mark.parametrize("io,out", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_norm_sizes(B, size, io, out):
    for kind in (B.LQ_NORM_RMS, B.LQ_NORM_MEAN):
        _check_norm(B, 5, 3, size, kind, B.LQ_ACT_SILU, True, False, False, True, True, io, out, seed=size)


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("gate", ["none", "after", "before"])
def test_norm_options(B, act, kind, gate):
    for shared, weight, bias in ((True, True, False), (False, True, True), (False, False, False)):
        _check_norm(B, 37, 5, 64, kind, act, gate != "none", gate == "before", shared, weight, bias, BF, F32)


@pytest.mark.parametrize("n,groups,size", [(1, 1, 128), (1, 32, 128), (9001, 32, 128), (40000, 1, 64), (2100, 33, 32),
                                           (700, 1000, 8), (3, 65535, 4)])
def test_norm_shapes(B, n, groups, size):
    _check_norm(B, n, groups, size, B.LQ_NORM_MEAN, B.LQ_ACT_SIGMOID, True, False, False, True, False, BF, BF)


def test_norm_unaligned_rows(B):
    for size in (128, 600):
        for io in (BF, F32):
            _check_norm(B, 33, 3, size, B.LQ_NORM_RMS, B.LQ_ACT_SILU, True, False, True, True, False, io, F32,
                        misalign=True)


def test_norm_in_place_and_values_that_are_not_finite(B):
    x = torch.randn((6, 4, 128), device="cuda")
    x[1, 2, 5], x[3, 0, 7] = math.nan, math.inf
    z = torch.randn((6, 4, 128), device="cuda")
    z[5, 1, :] = -200.0  # the sigmoid's far end
    cfg = B.make_norm_config(4, 128)
    y = torch.empty_like(x)
    B.lq_group_norm(cfg, 6, x, y, gate=z)
    bad = ~torch.isfinite(y).all(-1)
    want = torch.zeros((6, 4), dtype=torch.bool, device="cuda")
    want[1, 2] = want[3, 0] = True  # the groups that hold them, and no other
    assert torch.equal(bad, want)
    assert bool((y[5, 1] == 0).all())
    over_x, over_z = x.clone(), z.clone()
    B.lq_group_norm(cfg, 6, over_x, over_x, gate=z)
    B.lq_group_norm(cfg, 6, x, over_z, gate=over_z)
    for got in (over_x, over_z):
        assert torch.equal(got.nan_to_num(9.0), y.nan_to_num(9.0))


# ---------------------------------------------------------------------------
# Together, and next to the int8 decode path
# ---------------------------------------------------------------------------

def test_a_layer_prompt_then_tokens(B):
    """Rotary, the recurrence, the gated norm: a prompt in one call of each, and
    the same tokens one at a time from a graph, against 64 bits."""
    hk, hv, d, n, rot = 2, 4, 64, 90, 32
    g = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.randn((n, (2 * hk + 2 * hv) * d), generator=g, device="cuda")
    a, c = hk * d, hv * d
    cut = [rows[:, :a], rows[:, a:2 * a], rows[:, 2 * a:2 * a + c], rows[:, 2 * a + c:]]
    q, k, v, z = (x.unflatten(1, (-1, d)) for x in cut)
    stride = rows.stride(0)
    pos = torch.arange(1000, 1000 + n, dtype=torch.int32, device="cuda")
    decay = torch.exp(-torch.exp2(-8.0 * torch.arange(1, hv + 1, device="cuda") / hv))
    w = 1 + 0.1 * torch.randn((d,), generator=g, device="cuda")
    table, mag = B.lq_rotary_table(rot, 10000.0, B.LQ_ROPE_PARTS, 8.0, 4096.0)
    table = table.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def layer(tokens, q, k, v, z, pos, S, offsets):
        qr, kr = torch.empty((tokens, hk, d), device="cuda"), torch.empty((tokens, hk, d), device="cuda")
        o, y = torch.empty((tokens, hv, d), device="cuda"), torch.empty((tokens, hv, d), device="cuda")
        B.lq_rotary(B.make_rotary_config(hk, hk, d, rot, bf16=False, magnitude=mag, q_stride=stride,
                                         k_stride=stride), tokens, q, k, pos, table, qr, kr)
        cfg = B.make_linear_config(1, hk, hv, d, d, decay=B.LQ_DECAY_HEAD, v_stride=stride)
        if offsets is None:
            B.lq_linear_decode_step(cfg, qr, kr, v, decay, S, 1, o, err)
        else:
            ws = torch.empty(max(16, B.lq_linear_workspace_bytes(cfg, tokens)), dtype=torch.uint8, device="cuda")
            B.lq_linear_prefill(cfg, qr, kr, v, decay, tokens, offsets, S, 1, o, err, workspace=ws)
        B.lq_group_norm(B.make_norm_config(hv, d, shared_weight=True, gate_stride=stride), tokens, o, y, gate=z,
                        weight=w)
        return y

    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2 * i / rot)
    keep = ((4096.0 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
    f = f * keep + f / 8 * (1 - keep)

    def turned(x):
        return _rotated(x, pos, f, 0.1 * math.log(8.0) + 1, "half", rot, False)[0].repeat_interleave(hv // hk, 1)

    qd, kd, S64 = turned(q), turned(k), torch.zeros((hv, d, d), dtype=torch.float64, device="cuda")
    want = torch.empty((n, hv, d), dtype=torch.float64, device="cuda")
    for t in range(n):
        S64 = decay.double()[:, None, None] * S64 + v[t].double()[:, :, None] * kd[t][:, None, :]
        want[t] = torch.einsum("hvk,hk->hv", S64, qd[t])
    want = want / torch.sqrt((want ** 2).mean(-1, keepdim=True) + 1e-5) * w.double()
    want = want * z.double() * torch.sigmoid(z.double())

    S = torch.zeros((1, hv, d, d), device="cuda")
    y = layer(n, q, k, v, z, pos, S, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    # errors of 1e-6 a stage in quadrature, with a factor of 10
    assert float((y.double() - want).norm()) <= 2e-5 * float(want.norm())

    S2 = torch.zeros((1, hv, d, d), device="cuda")
    row, p1 = rows[:1].clone(), pos[:1].clone()
    parts = [x.unflatten(1, (-1, d)) for x in (row[:, :a], row[:, a:2 * a], row[:, 2 * a:2 * a + c], row[:, 2 * a + c:])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = layer(1, *parts, p1, S2, None)
    S2.zero_()
    got = torch.empty_like(y)
    for t in range(n):
        row.copy_(rows[t:t + 1])
        p1.copy_(pos[t:t + 1])
        graph.replay()
        got[t] = y1[0]
    assert float((got.double() - want).norm()) <= 2e-5 * float(want.norm())
    assert float((S2 - S).norm()) <= 2e-5 * float(S.norm())
    assert int(err) == 0


def test_norm_of_the_int8_decode_steps_outputs(B):
    """The norm takes lq_decode_step's [B][Hv][d] outputs as they are."""
    from recurrent_state_quantization_decode_b200 import workloads as wl

    import numpy as np

    w = wl.Workload("n", 3, 2, 4, 128, wl.GATE_SCALAR, True, 1)
    rng = np.random.default_rng(4)
    S0, _, _ = wl.initial_states(rng, w.tiles, w.d, w.d)
    ti = wl.token_inputs(rng, w, 1)
    cfg, out = B.config_for(w), torch.empty((3, 4, 128), device="cuda")
    ds = B.DeviceState(cfg)
    B.lq_state_init(cfg, torch.from_numpy(S0).cuda(), ds.st)
    dev = [torch.from_numpy(getattr(ti, x)[0]).cuda() for x in ("q", "k", "v", "alpha", "beta")]
    dev[:3] = [x.to(BF) for x in dev[:3]]
    B.lq_decode_step(cfg, *dev, ds.st, out)
    gate, wt = torch.randn((3, 4, 128), device="cuda"), torch.rand((128,), device="cuda") + 0.5
    y = torch.empty((3, 4, 128), dtype=BF, device="cuda")
    B.lq_group_norm(B.make_norm_config(4, 128, shared_weight=True, out_bf16=True), 3, out, y, gate=gate, weight=wt)
    o = out.double()
    want = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-5) * wt.double() * gate.double() * torch.sigmoid(
        gate.double())
    assert bool(((y.double() - want).abs() <= want.abs() * (R + 300 * U) + 1e-30).all())


# ---------------------------------------------------------------------------
# Linear attention: orders of the sequences
# ---------------------------------------------------------------------------

UNEVEN = [6000, 0, 3950, 130, 168, 127, 369, 381, 520, 2244, 165, 257, 211, 109, 197, 730, 779, 331, 943, 30, 183,
          744, 913, 530]  # the longest 1.4 shares of an SM at 32 heads: it stays whole


def _best_us(call):
    """The shortest of several runs of ten calls."""
    best = math.inf
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


@pytest.mark.parametrize("spare", [0, 120])
def test_prefill_orders(B, spare):
    """The order of the sequences changes no bit, and where the longest stands not the call's time: long
    ones start first (started last, the longest would add its whole time to the call's, 1.6 times as long
    in all)."""
    a = Linear(UNEVEN + [0] * spare, 16, 32, 128, 128, spare=0, seed=4)
    b = Linear([0] * spare + UNEVEN[1:] + UNEVEN[:1], 16, 32, 128, 128, spare=0, seed=4)
    order = list(range(len(UNEVEN), a.b)) + list(range(1, len(UNEVEN))) + [0]
    rows = torch.cat([torch.arange(a.off[i], a.off[i + 1], device="cuda") for i in order])
    b.q, b.k, b.v, b.decay = a.q[rows], a.k[rows], a.v[rows], a.decay[rows]
    b.S, b.slots = a.S, a.slots[torch.tensor(order, device="cuda")]
    took, got = [], []
    for c in (a, b):
        S, o = c.S.clone(), c.new_out()
        ws = c.prefill(B, S, o)
        got.append((S, o))
        S, o = c.S.clone(), c.new_out()
        took.append(_best_us(lambda: c.prefill(B, S, o, ws=ws)))
        assert int(c.err) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1][rows], got[1][1])
    assert took[1] <= 1.25 * took[0], took


def test_prefill_of_a_long_sequence_among_many(B):
    """More sequences than are ranked by length: a long one is cut wherever it stands."""
    lengths = [1] * 500 + [30000] + [1] * 400
    c = Linear(lengths, 1, 2, 64, 64, out=F32, spare=0, seed=6)
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o)
    one = Linear([30000], 1, 2, 64, 64, out=F32, spare=0)
    rows = slice(500, 30500)
    one.q, one.k, one.v, one.decay = c.q[rows], c.k[rows], c.v[rows], c.decay[rows]
    one.S, at = c.S[c.slots[500].long()][None].clone(), int(c.slots[500])
    S1, o1 = one.S.clone(), one.new_out()
    one.prefill(B, S1, o1)
    for got, want in ((o[rows], o1), (S[at], S1[0])):  # fp32 results, cut in other places
        assert float((got - want).norm()) <= 2e-5 * float(want.norm())
    # the others are single tokens
    rest = torch.cat([torch.arange(500, device="cuda"), torch.arange(30500, c.n, device="cuda")])
    ids = torch.cat([torch.arange(500, device="cuda"), torch.arange(501, c.b, device="cuda")])
    step = B.make_linear_config(900, 1, 2, 64, 64, in_bf16=True)
    S2, o2 = c.S.clone(), torch.empty((900, 2, 64), device="cuda")
    B.lq_linear_decode_step(step, c.q[rest], c.k[rest], c.v[rest], c.decay[rest], S2, c.num_slots, o2, c.err,
                            slots=c.slots[ids])
    used = c.slots[ids].long()
    assert float((o[rest] - o2).norm()) <= 2e-5 * float(o2.norm())
    assert float((S[used] - S2[used]).norm()) <= 2e-5 * float(S2[used].norm())
    assert int(c.err) == 0 and int(one.err) == 0


@pytest.mark.parametrize("io", [BF, F32])
def test_prefill_in_the_largest_calls_workspace(B, io):
    """One workspace, sized for the largest call, serves all smaller ones, and nothing behind it is written."""
    big = B.make_linear_config(6, 2, 8, 128, 128, in_bf16=io == BF)
    size = B.lq_linear_workspace_bytes(big, 4000)
    for lengths in ([129], [700], [1280], [1281], [2000, 1, 1999], [900, 0, 33, 1200, 7, 640], [4000]):
        c = Linear(lengths, 2, 8, 128, 128, io, F32, seed=len(lengths))
        ws = torch.full((size + (1 << 20),), 171, dtype=torch.uint8, device="cuda")
        S, o = c.S.clone(), c.new_out()
        c.prefill(B, S, o, ws=ws[:size])
        c.check(o, S)
        assert bool((ws[size:] == 171).all())


def test_rotary_of_the_most_tokens(B):
    """2^31 - 1 tokens of one head of two channels, in place."""
    n = (1 << 31) - 1
    q = torch.ones((n, 1, 2), dtype=BF, device="cuda")
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    moved = torch.tensor([0, 1, 7, 8, n // 2, n - 9, n - 8, n - 1], device="cuda")
    pos[moved] = torch.arange(1, 9, dtype=torch.int32, device="cuda")
    table, _ = B.lq_rotary_table(2)
    B.lq_rotary(B.make_rotary_config(1, 0, 2, 2), n, q, None, pos, table.cuda(), q, None)
    a = torch.arange(1, 9, dtype=torch.float64, device="cuda")
    want = torch.stack([torch.cos(a) - torch.sin(a), torch.cos(a) + torch.sin(a)], -1)
    d = (q[moved, 0].double() - want).abs()
    assert bool((d <= R * want.abs() + 32 * U).all())
    q[moved] = 1.0  # position 0 turns nothing
    for part in q.view(-1).split(1 << 28):
        assert bool((part == 1.0).all())


# ---------------------------------------------------------------------------
# Linear attention: alignments
# ---------------------------------------------------------------------------

def _inside(t, lead, fill):
    """(a copy of t that starts `lead` values into its allocation, the guards on both sides)."""
    n = t.numel()
    whole = torch.full((lead + n + 64,), fill, dtype=t.dtype, device="cuda")
    whole[lead:lead + n] = t.flatten()
    return whole[lead:lead + n].view(t.shape), (whole[:lead], whole[lead + n:])


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (32, 128)])
@pytest.mark.parametrize("io,out,lead", [(BF, BF, 1), (BF, BF, 8), (BF, F32, 1), (BF, F32, 4), (F32, F32, 1),
                                         (F32, BF, 3)])
def test_linear_alignments(B, dk, dv, io, out, lead):
    """Outputs at any whole value, states and the workspace at any 16 bytes: the same bits as from the start
    of an allocation, and nothing around them is written."""
    for lengths in ([1500], [300, 0, 128, 41, 700], [1] * 7):
        c = Linear(lengths, 1, 2, dk, dv, io, out, seed=dk + lead)
        S0, o0 = c.S.clone(), c.new_out()
        S1, around_S = _inside(c.S, 4, 5.0)
        o1, around_o = _inside(c.new_out(), lead, 7.0)
        if max(lengths) == 1:
            for S, o in ((S0, o0), (S1, o1)):
                B.lq_linear_decode_step(c.cfg(B), c.q, c.k, c.v, c.decay, S, c.num_slots, o, c.err, slots=c.slots)
        else:
            c.prefill(B, S0, o0)
            ws, around_ws = _inside(c.workspace(B, c.cfg(B)), 16, 171)
            c.prefill(B, S1, o1, ws=ws)
            assert all(bool((x == 171).all()) for x in around_ws)
        assert torch.equal(S0, S1) and torch.equal(o0, o1)
        assert all(bool((x == 5.0).all()) for x in around_S) and all(bool((x == 7.0).all()) for x in around_o)
        c.check(o1, S1)


# ---------------------------------------------------------------------------
# Linear attention: the roundings of bf16 outputs
# ---------------------------------------------------------------------------

def _check_roundings(c, out):
    """bf16 outputs of bf16 prompts round the output itself (r of it), and the state before the chunk and
    the decayed scores to two parts (2^-16 of the absolute terms); everything else is within the fp32
    bound u (2 * 128 + dk + 4) a chunk.  Value by value, and in the 2-norm with the output's rounding as
    random ones of r / sqrt(3)."""
    q, k, v, d = c.q.double(), c.k.double(), c.v.double(), c.decay.double()
    rep = c.hv // c.hk
    want, size = (torch.zeros((c.n, c.hv, c.dv), dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(c.b):
        S = c.S[int(c.slots[b])].double()
        if c.fresh is not None and int(c.fresh[b]):
            S = torch.zeros_like(S)
        A = S.abs()
        for t in range(c.off[b], c.off[b + 1]):
            a = d if c.decay_kind == "head" else d[t]
            kk, qq = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
            S = a[:, None, None] * S + v[t][:, :, None] * kk[:, None, :]
            A = a[:, None, None] * A + v[t].abs()[:, :, None] * kk.abs()[:, None, :]
            want[t] = torch.einsum("hvk,hk->hv", S, qq)
            size[t] = torch.einsum("hvk,hk->hv", A, qq.abs())
    chunks = -(-max(c.lengths) // 128)
    fine = (2.0 ** -16 + U * (256 + c.dk + 4) * chunks) * size
    do = (out[:c.n].double() - want).abs()
    lim = R * want.abs() * (1 + R) + fine + 1e-30
    assert bool((do <= lim).all()), float((do / lim).max())
    norm = R / math.sqrt(3) * float(want.norm()) + float(fine.norm())
    assert float(do.norm()) <= norm, (float(do.norm()), norm)


ROUNDINGS = {
    "first_chunk": dict(lengths=[128, 77, 1, 100], hk=2, hv=4, dk=128, dv=128),
    "first_chunk_d64": dict(lengths=[128, 50, 40], hk=1, hv=2, dk=64, dv=64, decay="head"),
    "carried": dict(lengths=[700, 129, 256], hk=1, hv=2, dk=128, dv=128),
    "slow": dict(lengths=[1500], hk=1, hv=2, dk=128, dv=64, decay="head"),
}


@pytest.mark.parametrize("name", sorted(ROUNDINGS))
def test_prefill_roundings_of_bf16_outputs(B, name):
    c = Linear(**ROUNDINGS[name], seed=21)
    if name.startswith("first"):
        c.fresh = torch.ones(c.b, dtype=torch.int32, device="cuda")
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o)
    assert int(c.err) == 0
    _check_roundings(c, o)


def test_prefill_rows_of_one_score(B):
    """Each output is one score's: nothing averages its roundings."""
    c = Linear([128, 128, 90], 1, 2, 128, 128, seed=22)
    c.fresh = torch.ones(c.b, dtype=torch.int32, device="cuda")
    eye = torch.eye(128, device="cuda")
    for b in range(c.b):
        t = torch.arange(c.lengths[b], device="cuda")
        c.k[c.off[b]:c.off[b + 1], 0] = eye[t].to(BF)
        c.q[c.off[b]:c.off[b + 1], 0] = eye[(t - 5 * b).clamp(min=0)].to(BF)
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o)
    assert int(c.err) == 0
    _check_roundings(c, o)


def test_prefill_of_a_state_nearly_orthogonal_to_q(B):
    """A large state of which q sees a small difference: roundings of the state's values would show in
    the outputs."""
    for out in (BF, F32):
        c = Linear([128, 300], 1, 2, 128, 128, out=out, seed=23)
        c.S = c.S * 50.0
        for b in range(c.b):
            S = c.S[int(c.slots[b])]
            S[:, :, 1::2] = -S[:, :, 0::2]  # q with equal pairs sees nothing of it
            q = c.q[c.off[b]:c.off[b + 1]]
            q[..., 1::2] = q[..., 0::2]
        S, o = c.S.clone(), c.new_out()
        c.prefill(B, S, o)
        if out == BF:
            assert int(c.err) == 0
            _check_roundings(c, o)
        else:
            eo, _ = c.exact()
            ao, _ = c.exact(absolute=True)
            assert bool(((o[:c.n].double() - eo).abs() <= U * (2 * 384 + 132) * ao + U * eo.abs()).all())


# ---------------------------------------------------------------------------
# Larger and odder calls
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("out", [BF, F32])
def test_prefill_of_short_bf16_sequences(B, dk, dv, out):
    """At most 32 tokens a sequence on average, a long one among them too: token by token, in segments."""
    for lengths in ([20, 1, 31, 0, 7], [333] + [0, 1] * 20):
        c = Linear(lengths, 2, 4, dk, dv, BF, out, fused=dv == 64, seed=dk * dv)
        c.fresh = (torch.arange(c.b) % 3 == 1).to(torch.int32).cuda()
        S, o = c.S.clone(), c.new_out()
        c.prefill(B, S, o)
        c.check(o, S)


@pytest.mark.parametrize("io", [BF, F32])
def test_prefill_faults_among_many_sequences(B, io):
    """More sequences than a warp looks at by itself: slots that cannot be used, and offsets past the rows."""
    lengths = [40 + i % 90 for i in range(150)]
    c = Linear(lengths, 1, 1, 32, 64, io, F32, seed=9)
    own = c.slots.clone()
    for change, report in (({149: -1, 3: -5}, False), ({140: int(own[0])}, True), ({0: c.num_slots, 131: 1 << 30}, True)):
        c.slots = own.clone()
        for i, s in change.items():
            c.slots[i] = s
        S, o = c.S.clone(), c.new_out()
        c.prefill(B, S, o)
        assert B.lq_get_error_word(c.err) == (B.LQ_ERR_DEVICE_BOUNDS if report else B.LQ_OK)
        c.check(o, S, skip=tuple(change))
    c.slots = own
    c.offsets[150] = c.n + 1
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o)
    assert B.lq_get_error_word(c.err) == B.LQ_ERR_DEVICE_BOUNDS
    c.check(o, S, skip=(149,))


@pytest.mark.parametrize("hk,hv,d,lengths", [(1, 640, 32, [300, 5]), (160, 160, 64, [150]), (7, 49, 32, [400, 129])])
def test_prefill_head_counts(B, hk, hv, d, lengths):
    """More heads than SMs, or none of their divisors."""
    for io in (BF, F32):
        c = Linear(lengths, hk, hv, d, d, io, F32, seed=hv)
        S, o = c.S.clone(), c.new_out()
        c.prefill(B, S, o)
        c.check(o, S)


@pytest.mark.parametrize("io,size", [(BF, 1 << 22), (F32, 1 << 21)])
def test_prefill_rows_past_32_bit_offsets(B, io, size):
    """Token rows so far apart that the last ones start more than 2^32 bytes and 2^30 values into them."""
    c = Linear([257, 0, 300], 1, 2, 64, 64, io, F32, seed=2)
    rows = torch.empty((c.n, size), dtype=io, device="cuda")
    rows[:, :64], rows[:, 64:128], rows[:, 128:256] = c.q[:, 0], c.k[:, 0], c.v.flatten(1)
    c.q, c.k, c.v = (rows[:, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 64), (64, 128), (128, 256)))
    S, o = c.S.clone(), c.new_out()
    c.prefill(B, S, o)
    c.check(o, S)


def test_norm_past_32_bit_offsets(B):
    """More than 2^31 values, in place."""
    n, groups, size = 66001, 32, 1024
    x = torch.ones((n, groups, size), dtype=BF, device="cuda")
    at = torch.tensor([0, 1, n // 2, 65535, 65536, n - 2, n - 1], device="cuda")
    some = torch.randn((len(at), groups, size), device="cuda").to(BF)
    x[at] = some
    B.lq_group_norm(B.make_norm_config(groups, size, act=B.LQ_ACT_NONE, in_bf16=True, out_bf16=True, eps=0.0), n, x, x)
    want = some.double() / torch.sqrt((some.double() ** 2).mean(-1, keepdim=True))
    d = (x[at].double() - want).abs()
    assert bool((d <= want.abs() * (R + (size + 12) * U)).all())
    x[at] = 1.0  # rows of ones stay ones
    for part in x.view(-1).split(1 << 28):
        assert bool((part == 1.0).all())
