"""The layer operators (include/leapquant_layer.h) without a GPU: the library
exports what the header declares, argument errors come back before anything is
launched, and the rotary table is the frequencies' definition."""
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def B():
    from recurrent_state_quantization_decode_b200 import build

    build.build()
    from recurrent_state_quantization_decode_b200 import binding

    return binding


def _status(B, fn, *args, **kw):
    with pytest.raises(B.LQError) as ei:
        fn(*args, stream=0, **kw) if fn is not B.lq_rotary_table else fn(*args, **kw)
    return ei.value.status


def test_exports_every_declared_symbol(B):
    txt = open(os.path.join(ROOT, "include", "leapquant_layer.h")).read()
    names = sorted(set(re.findall(r"\b(lq_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", txt, flags=re.S))))
    assert sorted(B.EXPORTED_LAYER) == names
    for n in names:
        assert hasattr(B._lib, n), n


def _step(B, cfg, q=GOOD, k=GOOD, v=GOOD, decay=GOOD, S=GOOD, n=4, out=GOOD, err=GOOD, slots=None):
    B.lq_linear_decode_step(cfg, q, k, v, decay, S, n, out, err, slots=slots, stream=0)


def _prefill(B, cfg, q=GOOD, k=GOOD, v=GOOD, decay=GOOD, tokens=8, offsets=GOOD, S=GOOD, n=4, out=GOOD,
             err=GOOD, **kw):
    B.lq_linear_prefill(cfg, q, k, v, decay, tokens, offsets, S, n, out, err, stream=0, **kw)


@pytest.mark.parametrize("field,value,status", [
    ("batch", -1, 1), ("num_k_heads", 0, 1), ("num_v_heads", 3, 1), ("decay", 2, 1), ("in_dtype", 2, 1),
    ("out_dtype", -1, 1), ("dk", 96, 2), ("dv", 256, 2), ("dk", 0, 2), ("batch", 1 << 19, 2),
    ("num_k_heads", 4096, 2), ("q_stride", -128, 1), ("k_stride", 64, 1), ("v_stride", 256, 1),
    ("q_stride", 130, 3), ("v_stride", 514, 3),
])
def test_linear_config_is_checked(B, field, value, status):
    cfg = B.make_linear_config(2, 2, 4, 64, 128)
    setattr(cfg, field, value)
    if (field, value) == ("num_k_heads", 4096):
        cfg.num_v_heads = 4096
    for call in (_step, _prefill):
        with pytest.raises(B.LQError) as ei:
            call(B, cfg)
        assert ei.value.status == status
    assert B.lq_linear_workspace_bytes(cfg, 100) == 0


def test_linear_batch_has_a_limit(B):
    """The blocks' work on slots and lengths grows with the batch's square."""
    cfg = B.make_linear_config(65536, 1, 1, 64, 64)
    assert B.lq_linear_workspace_bytes(cfg, 1 << 24) > 0
    cfg.batch = 65537
    assert B.lq_linear_workspace_bytes(cfg, 1 << 24) == 0
    for call in (_step, _prefill):
        with pytest.raises(B.LQError) as ei:
            call(B, cfg)
        assert ei.value.status == B.LQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(decay=None), 1), (dict(S=None), 1),
    (dict(err=None), 1), (dict(n=-1), 1), (dict(n=1), 1), (dict(q=GOOD + 8), 3), (dict(k=GOOD + 2), 3),
    (dict(v=GOOD + 4), 3), (dict(decay=GOOD + 2), 3), (dict(S=GOOD + 4), 3), (dict(out=GOOD + 1), 3),
    (dict(err=GOOD + 2), 3), (dict(slots=GOOD + 2), 3),
])
def test_linear_pointers_are_checked(B, kw, status):
    cfg = B.make_linear_config(2, 2, 4, 64, 64, in_bf16=True, out_bf16=True)
    for call in (_step, _prefill):
        with pytest.raises(B.LQError) as ei:
            call(B, cfg, **kw)
        assert ei.value.status == status


def test_linear_calls_of_their_own_checks(B):
    cfg = B.make_linear_config(2, 2, 4, 64, 64)
    with pytest.raises(B.LQError) as ei:
        _step(B, cfg, out=None)
    assert ei.value.status == B.LQ_ERR_INVALID_ARG
    for kw, status in ((dict(tokens=-1), 1), (dict(offsets=None), 1), (dict(offsets=GOOD + 2), 3),
                       (dict(fresh=GOOD + 1), 3), (dict(workspace=GOOD + 8), 3)):
        with pytest.raises(B.LQError) as ei:
            _prefill(B, cfg, **kw)
        assert ei.value.status == status, kw
    # a workspace that is asked for and too small, or missing, is refused
    big = B.make_linear_config(2, 2, 4, 128, 128, in_bf16=True)
    need = B.lq_linear_workspace_bytes(big, 1 << 20)
    if need:
        for w in (None, torch.empty(0)):
            with pytest.raises((B.LQError, ValueError)):
                _prefill(B, big, tokens=1 << 20, workspace=w)
    # an empty batch is a valid call
    empty = B.make_linear_config(0, 2, 4, 64, 64)
    _step(B, empty)
    _prefill(B, empty, tokens=0, q=None, k=None, v=None, decay=None)


def _rotary(B, cfg, tokens=4, q=GOOD, k=GOOD, positions=GOOD, table=GOOD, q_out=2 * GOOD, k_out=2 * GOOD):
    B.lq_rotary(cfg, tokens, q, k, positions, table, q_out, k_out, stream=0)


def test_rotary_arguments_are_checked(B):
    def cfg(**kw):
        c = B.make_rotary_config(4, 2, 64, 64)
        for f, x in kw.items():
            setattr(c, f, x)
        return c

    for fields, status in ((dict(rot=63), 1), (dict(rot=0), 1), (dict(rot=66), 1), (dict(layout=2), 1),
                           (dict(dtype=3), 1), (dict(num_q_heads=-1), 1), (dict(d=2048, rot=64), 2),
                           (dict(num_q_heads=65535), 2), (dict(q_stride=128), 1), (dict(k_out_stride=-1), 1)):
        with pytest.raises(B.LQError) as ei:
            _rotary(B, cfg(**fields))
        assert ei.value.status == status, fields
    for kw, status in ((dict(tokens=-1), 1), (dict(q=None), 1), (dict(k_out=None), 1), (dict(positions=None), 1),
                       (dict(table=None), 1), (dict(q=GOOD + 1), 3), (dict(table=GOOD + 4), 3),
                       (dict(positions=GOOD + 2), 3)):
        with pytest.raises(B.LQError) as ei:
            _rotary(B, cfg(), **kw)
        assert ei.value.status == status, kw
    with pytest.raises(B.LQError) as ei:  # in place with another stride
        _rotary(B, cfg(q_stride=512), q_out=GOOD)
    assert ei.value.status == B.LQ_ERR_INVALID_ARG
    _rotary(B, cfg(), tokens=0)
    _rotary(B, cfg(num_q_heads=0, num_k_heads=0))


def test_norm_arguments_are_checked(B):
    def call(x=GOOD, out=2 * GOOD, tokens=4, gate=None, weight=None, bias=None, **fields):
        c = B.make_norm_config(4, 32)
        for f, v in fields.items():
            setattr(c, f, v)
        B.lq_group_norm(c, tokens, x, out, gate=gate, weight=weight, bias=bias, stream=0)

    for kw, status in ((dict(groups=0), 1), (dict(size=0), 1), (dict(size=8193), 2), (dict(groups=65536), 2),
                       (dict(kind=2), 1), (dict(act=3), 1), (dict(in_dtype=2), 1), (dict(out_dtype=2), 1),
                       (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x_stride=127), 1),
                       (dict(out_stride=-1), 1), (dict(gate_before=1), 1), (dict(x=None), 1), (dict(out=None), 1),
                       (dict(tokens=-1), 1), (dict(tokens=1 << 30), 2), (dict(x=GOOD + 2), 3),
                       (dict(gate=GOOD + 2), 3), (dict(weight=GOOD + 2), 3), (dict(bias=GOOD + 1), 3),
                       (dict(out=GOOD, x_stride=256), 1), (dict(out=GOOD, out_dtype=1), 1),
                       (dict(gate=2 * GOOD, gate_stride=256), 1)):
        with pytest.raises(B.LQError) as ei:
            call(**kw)
        assert ei.value.status == status, kw
    call(tokens=0)


def test_tensors_off_the_device_are_refused(B):
    cfg = B.make_norm_config(2, 16)
    with pytest.raises(ValueError):
        B.lq_group_norm(cfg, 1, torch.zeros(1, 2, 16), torch.zeros(1, 2, 16), stream=0)
    assert B.lq_get_error_word(0, 0) == B.LQ_ERR_INVALID_ARG


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts"])
@pytest.mark.parametrize("rot", [2, 14, 64, 128])
def test_rotary_table_is_the_frequencies(B, rot, scaling):
    """Entry i is f_i / 2 pi as a fraction of 2^64: with f_i in 64-bit floating
    point (relative error of a few 2^-53) the entries agree to 2^-46."""
    theta, factor, trained, fast, slow = 1e6, 8.0, 4096.0, 32.0, 1.0
    kind = {"none": B.LQ_ROPE_NONE, "linear": B.LQ_ROPE_LINEAR, "ntk": B.LQ_ROPE_NTK,
            "parts": B.LQ_ROPE_PARTS}[scaling]
    table, mag = B.lq_rotary_table(rot, theta, kind, factor, trained, fast, slow)
    assert table.shape == (rot // 2,)
    assert mag == pytest.approx(0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0, rel=1e-7)
    for i in range(rot // 2):
        base = theta * factor ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else theta
        f = math.exp(-2.0 * i / rot * math.log(base))
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            w = min(1.0, max(0.0, (trained * f / (2 * math.pi) - slow) / (fast - slow)))
            f = w * f + (1 - w) * f / factor
        want = f / (2 * math.pi) * 2.0 ** 64
        got = int(table[i]) % (1 << 64)
        assert abs(got - want) <= want * 2.0 ** -46 + 1, i  # exp(log) of 1e6: 14 * 2^-53 and the powers' own
        assert got <= 1 << 63


def test_rotary_table_arguments_are_checked(B):
    for args in ((63,), (0,), (64, 0.5), (64, float("inf")), (64, 1e4, 4), (64, 1e4, 1, 0.5),
                 (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 100.0, 1.0, 2.0)):
        assert _status(B, B.lq_rotary_table, *args) == B.LQ_ERR_INVALID_ARG, args
    assert _status(B, B.lq_rotary_table, 2048) == B.LQ_ERR_UNSUPPORTED


def _accepts(B, cfg, tokens, space):
    """Whether a prompt call takes a workspace of `space` bytes.  Without sequences it ends behind that
    check: nothing is launched."""
    empty = type(cfg).from_buffer_copy(cfg)
    empty.batch = 0
    status = B._lib.lq_linear_prefill(empty, GOOD, GOOD, GOOD, GOOD, tokens, GOOD, GOOD, 0, None, None, GOOD, GOOD,
                                      space, GOOD, None)
    assert status in (B.LQ_OK, B.LQ_ERR_INVALID_ARG)
    return status == B.LQ_OK


@pytest.mark.parametrize("hv,d,bf16", [(1, 128, True), (8, 128, True), (32, 128, True), (200, 32, True),
                                       (600, 64, True), (1, 64, False), (8, 64, False), (32, 128, False),
                                       (300, 32, False)])
def test_workspace_of_the_largest_call_is_enough(B, hv, d, bf16):
    """No smaller call, in tokens or in sequences, asks for more or is refused with the largest one's."""
    def size(batch, tokens):
        return B.lq_linear_workspace_bytes(B.make_linear_config(batch, hv, hv, d, d, in_bf16=bf16), tokens)

    counts = sorted({0, 1, 32, 33, 63, 64, 127, 128, 129, 130, 10368, 10369} | {17 * i for i in range(1, 900)}
                    | {128 * i + j for i in (5, 9, 81, 256, 1000, 5000) for j in (-1, 0, 1)}
                    | {1 << 20, (1 << 29) - 1, 1 << 29, 1 << 30, (1 << 31) - 1})
    for batch in (1, 2, 4, 24, 144, 1000):
        sizes = [size(batch, n) for n in counts]
        assert sizes == sorted(sizes), (batch, [n for n, a, b in zip(counts[1:], sizes, sizes[1:]) if b < a][:5])
    for n in counts:
        sizes = [size(b, n) for b in (1, 2, 3, 24, 144, 1000, 65536)]
        assert sizes == sorted(sizes), n
    cfg = B.make_linear_config(1, hv, hv, d, d, in_bf16=bf16)
    for n in counts:
        assert _accepts(B, cfg, n, size(1, n)), n


def test_workspace_below_the_need_is_refused(B):
    """One byte less than what a call needs, found by halving, is an argument error."""
    cfg = B.make_linear_config(1, 8, 8, 128, 128, in_bf16=True)
    for n in (8192, 20000, 1 << 20):
        least, most = 0, B.lq_linear_workspace_bytes(cfg, n)
        assert most > 0 and _accepts(B, cfg, n, most) and not _accepts(B, cfg, n, 0)
        while most - least > 1:
            half = (least + most) // 2
            least, most = (least, half) if _accepts(B, cfg, n, half) else (half, most)
        assert most % (8 * (128 * 128 + 1) * 4) == 0  # whole states and decays of 8 heads
        assert not _accepts(B, cfg, n, most - 1)


class _Fake:
    """A library that launches nothing and takes every call."""

    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def on_host(B, monkeypatch):
    """The binding with host tensors taken for the current device's, and no library behind it."""
    B._current()
    monkeypatch.setattr(B, "_lib", _Fake())
    monkeypatch.setattr(B, "_current", lambda: (-1, None))
    return B


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _refused(call, good, bad):
    """Takes the good arguments and refuses each changed one by its name."""
    call(**good)
    for name, x in bad:
        with pytest.raises(ValueError, match=rf"^{name}: "):
            call(**{**good, name: x})
    call(**good)


@pytest.mark.parametrize("head", [False, True])
def test_linear_tensors_of_another_type_or_too_small_are_refused(on_host, head):
    B, T, n, hk, hv, dk, dv = on_host, 9, 3, 2, 4, 32, 64
    cfg = B.make_linear_config(n, hk, hv, dk, dv, in_bf16=True,
                               decay=B.LQ_DECAY_HEAD if head else B.LQ_DECAY_TOKEN)
    rows = _bf(T, 2 * hk * dk + hv * dv)
    fused = B.make_linear_config(n, hk, hv, dk, dv, in_bf16=True, q_stride=rows.stride(0),
                                 k_stride=rows.stride(0), v_stride=rows.stride(0),
                                 decay=B.LQ_DECAY_HEAD if head else B.LQ_DECAY_TOKEN)

    def cut(r):
        a = hk * dk
        return dict(q=r[:, :a].unflatten(1, (hk, dk)), k=r[:, a:2 * a].unflatten(1, (hk, dk)),
                    v=r[:, 2 * a:].unflatten(1, (hv, dv)))

    def inputs(tokens):
        return dict(q=_bf(tokens, hk, dk), k=_bf(tokens, hk, dk), v=_bf(tokens, hv, dv),
                    decay=torch.zeros((hv,) if head else (tokens, hv)), S=torch.zeros(5, hv, dv, dk),
                    out=torch.zeros(tokens, hv, dv), err=torch.zeros(1, dtype=torch.int32),
                    slots=torch.zeros(n, dtype=torch.int32))

    def bad(tokens, good):
        return [("q", good["q"].float()), ("k", good["k"].half()), ("v", good["v"].float()),
                ("q", _bf(tokens - 1, hk, dk)), ("k", _bf(tokens, hk - 1, dk)), ("v", _bf(tokens - 1, hv, dv)),
                ("decay", good["decay"].double()), ("decay", good["decay"].flatten()[:-1]),
                ("S", good["S"].bfloat16()), ("S", good["S"][:4]), ("out", good["out"].bfloat16()),
                ("out", good["out"][:-1]), ("err", good["err"].long()), ("err", good["err"][:0]),
                ("slots", good["slots"].long()), ("slots", good["slots"][:-1])]

    def step(c=cfg, **kw):
        B.lq_linear_decode_step(c, num_slots=5, **kw)

    def prefill(c=cfg, **kw):
        B.lq_linear_prefill(c, tokens=T, num_slots=5, **kw)

    _refused(step, inputs(n), bad(n, inputs(n)))
    good = inputs(T)
    good.update(offsets=torch.zeros(n + 1, dtype=torch.int32), fresh=torch.zeros(n, dtype=torch.int32),
                workspace=torch.zeros(16, dtype=torch.uint8))
    _refused(prefill, good, bad(T, good) + [
        ("offsets", good["offsets"].long()), ("offsets", good["offsets"][:-1]), ("fresh", good["fresh"].bool()),
        ("fresh", good["fresh"][:-1])])
    # slices of a fused projection's rows: enough of them, and nothing past the last one's end
    good.update(cut(rows))
    prefill(c=fused, **good)
    for name, x in cut(rows[:-1]).items():
        with pytest.raises(ValueError, match=rf"^{name}: "):
            prefill(c=fused, **{**good, name: x})
    # other views of as many rows
    packed = inputs(T)
    packed.update(offsets=good["offsets"], q=_bf(T, hk * dk), k=_bf(T * hk * dk), v=_bf(1, T, hv, dv))
    prefill(**packed)
    prefill(**{**packed, "v": _bf(1, T + 1, hv, dv)})
    with pytest.raises(ValueError, match="^v: "):
        prefill(**{**packed, "v": _bf(1, T - 1, hv, dv)})


def test_rotary_tensors_of_another_type_or_too_small_are_refused(on_host):
    B, T = on_host, 5
    cfg = B.make_rotary_config(4, 2, 64, 32)
    good = dict(q=_bf(T, 4, 64), k=_bf(T, 2, 64), positions=torch.zeros(T, dtype=torch.int32),
                table=torch.zeros(16, dtype=torch.int64), q_out=_bf(T, 4, 64), k_out=_bf(T, 2, 64))
    _refused(lambda **kw: B.lq_rotary(cfg, T, **kw), good, [
        ("q", good["q"].float()), ("k", good["k"][:-1]), ("positions", good["positions"].long()),
        ("positions", good["positions"][:-1]), ("table", good["table"].int()), ("table", good["table"][:-1]),
        ("q_out", good["q_out"].half()), ("k_out", good["k_out"][:, :1])])
    B.lq_rotary(cfg, T, **{**good, "table": good["table"].view(torch.uint64)})
    # what a configuration without k heads does not look at
    B.lq_rotary(B.make_rotary_config(4, 0, 64, 32), T, **{**good, "k": torch.zeros(1), "k_out": None})


def test_norm_tensors_of_another_type_or_too_small_are_refused(on_host):
    B, T = on_host, 5
    good = dict(x=_bf(T, 3, 20), out=torch.zeros(T, 3, 20), gate=_bf(T, 3, 20), weight=torch.zeros(3, 20),
                bias=torch.zeros(3, 20))
    cfg = B.make_norm_config(3, 20, in_bf16=True)
    _refused(lambda **kw: B.lq_group_norm(cfg, T, **kw), good, [
        ("x", good["x"].float()), ("x", good["x"][:-1]), ("out", good["out"].bfloat16()), ("out", good["out"][:-1]),
        ("gate", good["gate"].float()), ("gate", good["gate"][:-1]), ("weight", good["weight"].bfloat16()),
        ("weight", good["weight"][0]), ("bias", good["bias"].double()), ("bias", good["bias"][0])])
    shared = B.make_norm_config(3, 20, in_bf16=True, shared_weight=True)
    B.lq_group_norm(shared, T, **{**good, "weight": good["weight"][0].clone()})
    with pytest.raises(ValueError, match="^err: "):
        B.lq_get_error_word(torch.zeros(1))
