"""Thin ctypes binding of libleapquant.so (include/leapquant.h).

Argument marshalling only: every step of the decode path runs in the library's
CUDA kernels.  Tensors are passed as device pointers (torch tensors are
accepted and must already live on the GPU, contiguous); PyTorch provides the
memory and the streams.  Importing this module fails loudly if the library
has not been built (python -m recurrent_state_quantization_decode_b200.build).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libleapquant.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python -m recurrent_state_quantization_decode_b200.build` (needs nvcc). "
        "There is no CPU fallback.")

_lib = ctypes.CDLL(LIB_PATH)

LQ_OK, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED, LQ_ERR_MISALIGNED, LQ_ERR_CUDA, \
    LQ_ERR_DEVICE_BOUNDS, LQ_ERR_TOO_LARGE, LQ_ERR_TIMEOUT = range(8)
LQ_NOALLOC_STAGING_MAX_BYTES = 8 << 20  # the fixed staging array of the no-alloc entry point
LQ_GATE_SCALAR, LQ_GATE_DIAG = 0, 1
LQ_DTYPE_F32, LQ_DTYPE_BF16 = 0, 1

# Every symbol include/leapquant.h declares.
EXPORTED = ("lq_version", "lq_status_string", "lq_state_layout", "lq_state_bytes",
            "lq_state_init", "lq_decode_step", "lq_decode_step_host",
            "lq_decode_step_host_noalloc", "lq_window_flush",
            "lq_fp32_decode_step", "lq_state_dequantize", "lq_get_last_error",
            "lq_test_decode_step_timeout", "lq_prefill", "lq_checkpoint_save",
            "lq_checkpoint_restore", "lq_window_rewind", "lq_decode_tokens",
            "lq_decode_step_packed")

LQ_DECAY_TOKEN, LQ_DECAY_HEAD = 0, 1
LQ_ROPE_HALF, LQ_ROPE_INTERLEAVED = 0, 1
LQ_ROPE_NONE, LQ_ROPE_LINEAR, LQ_ROPE_NTK, LQ_ROPE_PARTS = range(4)
LQ_NORM_RMS, LQ_NORM_MEAN = 0, 1
LQ_ACT_NONE, LQ_ACT_SILU, LQ_ACT_SIGMOID = range(3)

# Every symbol include/leapquant_layer.h declares.
EXPORTED_LAYER = ("lq_linear_decode_step", "lq_linear_workspace_bytes", "lq_linear_prefill",
                  "lq_rotary_table", "lq_rotary", "lq_group_norm", "lq_get_error_word")


class lq_config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_k_heads", ctypes.c_int32),
                ("num_v_heads", ctypes.c_int32), ("d", ctypes.c_int32),
                ("window", ctypes.c_int32), ("n_comp", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("smooth", ctypes.c_float)]


class lq_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "record_bytes", "off_sigma", "off_m", "off_comp_vec", "off_comp_id", "records_bytes",
        "buf_k_bytes", "buf_d_bytes", "buf_g_bytes", "buf_n_bytes", "err_bytes",
        "fp32_state_bytes", "host_staging_bytes")]


class lq_state(ctypes.Structure):
    _fields_ = [("records", ctypes.c_void_p), ("buf_k", ctypes.c_void_p),
                ("buf_d", ctypes.c_void_p), ("buf_g", ctypes.c_void_p),
                ("buf_n", ctypes.c_void_p), ("err", ctypes.c_void_p)]


class lq_linear_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_k_heads", "num_v_heads", "dk", "dv", "decay", "in_dtype", "out_dtype")] + \
        [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")]


class lq_rotary_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_q_heads", "num_k_heads", "d", "rot", "layout", "dtype", "inverse")] + \
        [("magnitude", ctypes.c_float)] + \
        [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")]


class lq_norm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "groups", "size", "kind", "act", "gate_before", "shared_weight", "in_dtype",
        "out_dtype")] + [("eps", ctypes.c_float)] + \
        [(n, ctypes.c_int64) for n in ("x_stride", "gate_stride", "out_stride")]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_F64 = ctypes.c_double
_LIN = ctypes.POINTER(lq_linear_config)
_ROT = ctypes.POINTER(lq_rotary_config)
_NORM = ctypes.POINTER(lq_norm_config)
_CFG = ctypes.POINTER(lq_config)
_ST = ctypes.POINTER(lq_state)
_sig = {
    "lq_version": ([], ctypes.c_int32),
    "lq_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "lq_state_layout": ([_CFG, ctypes.POINTER(lq_layout)], ctypes.c_int),
    "lq_state_bytes": ([_CFG, ctypes.POINTER(ctypes.c_size_t),
                        ctypes.POINTER(ctypes.c_size_t)], ctypes.c_size_t),
    "lq_state_init": ([_CFG, _P, _ST, _P, _P], ctypes.c_int),
    "lq_decode_step": ([_CFG, _P, _P, _P, _P, _P, _ST, _P, _P, _P], ctypes.c_int),
    "lq_decode_step_packed": ([_CFG, _P, _P, _P, _ST, _P, _P, _P], ctypes.c_int),
    "lq_decode_step_host": ([_CFG, _P, _P, _P, _P, _P, _ST, _P, _P, _P, _P], ctypes.c_int),
    "lq_decode_step_host_noalloc": ([_CFG, _P, _P, _P, _P, _P, _ST, _P, _P, _P], ctypes.c_int),
    "lq_window_flush": ([_CFG, _ST, _P, _P], ctypes.c_int),
    "lq_fp32_decode_step": ([_CFG, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "lq_state_dequantize": ([_CFG, _ST, ctypes.c_int32, _P, _P], ctypes.c_int),
    "lq_get_last_error": ([_ST, _P], ctypes.c_int),
    "lq_test_decode_step_timeout": ([_CFG, _P, _P, _P, _P, _P, _ST, _P, ctypes.c_uint32, _P],
                                    ctypes.c_int),
    "lq_prefill": ([_CFG, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _ST, _P, _P, _P],
                   ctypes.c_int),
    "lq_checkpoint_save": ([_CFG, _ST, _P, _P, ctypes.c_int32, _P], ctypes.c_int),
    "lq_checkpoint_restore": ([_CFG, _P, ctypes.c_int32, _P, _ST, _P], ctypes.c_int),
    "lq_window_rewind": ([_CFG, _ST, _P, _P], ctypes.c_int),
    "lq_decode_tokens": ([_CFG, ctypes.c_int32, _P, _P, _P, _P, _P, _ST, _P, _P, _P],
                         ctypes.c_int),
    "lq_linear_decode_step": ([_LIN, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P], ctypes.c_int),
    "lq_linear_workspace_bytes": ([_LIN, _I], ctypes.c_size_t),
    "lq_linear_prefill": ([_LIN, _P, _P, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, ctypes.c_size_t,
                           _P, _P], ctypes.c_int),
    "lq_rotary_table": ([_I, _F64, _I, _F64, _F64, _F64, _F64, _P,
                         ctypes.POINTER(ctypes.c_float)], ctypes.c_int),
    "lq_rotary": ([_ROT, _I, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "lq_group_norm": ([_NORM, _I, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "lq_get_error_word": ([_P, _P], ctypes.c_int),
}
for _name, (_args, _res) in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class LQError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {lq_status_string(status)}")


def _check(status: int, call: str) -> None:
    if status != LQ_OK:
        raise LQError(status, call)


def _ptr(x) -> Optional[int]:
    """Device (or host) address of a tensor / int / None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if hasattr(x, "is_contiguous") and not x.is_contiguous():
            raise ValueError("tensors passed to libleapquant must be contiguous")
        return x.data_ptr()
    raise TypeError(f"cannot pass {type(x).__name__} as a pointer")


def _stream(stream) -> Optional[int]:
    if stream is None:
        try:
            import torch
            if torch.cuda.is_available():
                return torch.cuda.current_stream().cuda_stream
        except ImportError:
            pass
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_config(batch: int, num_k_heads: int, num_v_heads: int, d: int, window: int = 16,
                n_comp: int = 4, gate: int = LQ_GATE_SCALAR, in_bf16: bool = False,
                out_bf16: bool = False, smooth: float = 0.5) -> lq_config:
    return lq_config(batch, num_k_heads, num_v_heads, d, window, n_comp, gate,
                     LQ_DTYPE_BF16 if in_bf16 else LQ_DTYPE_F32,
                     LQ_DTYPE_BF16 if out_bf16 else LQ_DTYPE_F32, smooth)


def config_for(workload, batch: Optional[int] = None, out_bf16: bool = False) -> lq_config:
    """lq_config of a workloads.Workload."""
    w = workload
    return make_config(w.batch if batch is None else batch, w.num_k_heads, w.num_v_heads, w.d,
                       w.window, w.n_comp, w.gate, w.io_bf16, out_bf16, w.smooth)


# ---------------------------------------------------------------------------
# The C entry points, same names
# ---------------------------------------------------------------------------

def lq_version() -> int:
    return _lib.lq_version()


def lq_status_string(status: int) -> str:
    return _lib.lq_status_string(status).decode()


def lq_state_layout(cfg: lq_config) -> lq_layout:
    out = lq_layout()
    _check(_lib.lq_state_layout(ctypes.byref(cfg), ctypes.byref(out)), "lq_state_layout")
    return out


def lq_state_bytes(cfg: lq_config) -> tuple[int, int, int]:
    """(total, tile_bytes, buffer_bytes); total 0 means a bad cfg."""
    tb, bb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    total = _lib.lq_state_bytes(ctypes.byref(cfg), ctypes.byref(tb), ctypes.byref(bb))
    return total, tb.value, bb.value


def lq_state_init(cfg, S0, state: lq_state, mask=None, stream=None) -> None:
    _check(_lib.lq_state_init(ctypes.byref(cfg), _ptr(S0), ctypes.byref(state), _ptr(mask),
                              _stream(stream)), "lq_state_init")


def lq_decode_step(cfg, q, k, v, alpha, beta, state: lq_state, out, active=None,
                   stream=None) -> None:
    _check(_lib.lq_decode_step(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                               _ptr(beta), ctypes.byref(state), _ptr(out), _ptr(active),
                               _stream(stream)), "lq_decode_step")


def lq_decode_step_packed(cfg, qkva, alpha, beta, state: lq_state, out, active=None,
                          stream=None) -> None:
    """lq_decode_step with each tile's q, k, v (and KDA gate) packed back to
    back in qkva (see pack_tile_inputs); alpha: the GDN gates, None for KDA."""
    _check(_lib.lq_decode_step_packed(ctypes.byref(cfg), _ptr(qkva), _ptr(alpha), _ptr(beta),
                                      ctypes.byref(state), _ptr(out), _ptr(active),
                                      _stream(stream)), "lq_decode_step_packed")


def pack_tile_inputs(cfg, q, k, v, alpha):
    """The per-tile block layout of lq_decode_step_packed from q, k [B][Hk][d],
    v [B][Hv][d] and, for KDA, alpha [B][Hv][d] (torch tensors on one device):
    a uint8 tensor [B][Hv][block bytes]."""
    import torch

    B, Hk, Hv = cfg.batch, cfg.num_k_heads, cfg.num_v_heads
    g = Hv // Hk
    parts = [q.repeat_interleave(g, dim=1), k.repeat_interleave(g, dim=1), v]
    blocks = [x.contiguous().view(torch.uint8).reshape(B, Hv, -1) for x in parts]
    if cfg.gate == LQ_GATE_DIAG:
        blocks.append(alpha.contiguous().view(torch.uint8).reshape(B, Hv, -1))
    return torch.cat(blocks, dim=2).contiguous()


def lq_decode_tokens(cfg, ntok: int, q, k, v, alpha, beta, state: lq_state, out, active=None,
                     stream=None) -> None:
    """ntok consecutive decode tokens in one launch (token-major inputs and
    outputs, each token laid out as for lq_decode_step)."""
    _check(_lib.lq_decode_tokens(ctypes.byref(cfg), ctypes.c_int32(ntok), _ptr(q), _ptr(k),
                                 _ptr(v), _ptr(alpha), _ptr(beta), ctypes.byref(state),
                                 _ptr(out), _ptr(active), _stream(stream)), "lq_decode_tokens")


def lq_prefill(cfg, q, k, v, alpha, beta, T: int, S0, state: lq_state, out=None, mask=None,
               stream=None) -> None:
    """Exact recurrence over a T-token prompt (token-major inputs), outputs to
    `out` ([T, B, Hv, d], optional), then the quantizer into `state`."""
    _check(_lib.lq_prefill(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                           _ptr(beta), ctypes.c_int32(T), _ptr(S0), ctypes.byref(state),
                           _ptr(out), _ptr(mask), _stream(stream)), "lq_prefill")


def lq_checkpoint_save(cfg, state: lq_state, slots, pool, num_slots: int,
                       stream=None) -> None:
    """Copy the records of the sequences with slots[b] >= 0 into pool slot
    slots[b] (tiles must be on a window boundary)."""
    _check(_lib.lq_checkpoint_save(ctypes.byref(cfg), ctypes.byref(state), _ptr(slots),
                                   _ptr(pool), ctypes.c_int32(num_slots), _stream(stream)),
           "lq_checkpoint_save")


def lq_checkpoint_restore(cfg, pool, num_slots: int, slots, state: lq_state,
                          stream=None) -> None:
    """Copy pool slot slots[b] into sequence b's records (buf_n = 0)."""
    _check(_lib.lq_checkpoint_restore(ctypes.byref(cfg), _ptr(pool), ctypes.c_int32(num_slots),
                                      _ptr(slots), ctypes.byref(state), _stream(stream)),
           "lq_checkpoint_restore")


def lq_window_rewind(cfg, state: lq_state, drop, stream=None) -> None:
    """Drop the last drop[b] decoded tokens of sequence b (inside a window)."""
    _check(_lib.lq_window_rewind(ctypes.byref(cfg), ctypes.byref(state), _ptr(drop),
                                 _stream(stream)), "lq_window_rewind")


def lq_test_decode_step_timeout(cfg, q, k, v, alpha, beta, state: lq_state, out,
                                wait_limit: int, stream=None) -> None:
    """Testing only: lq_decode_step in which the first CTA withholds the copies
    of its first ring slot, so that its bounded wait (wait_limit polls) expires
    and the error word reports LQ_ERR_TIMEOUT."""
    _check(_lib.lq_test_decode_step_timeout(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v),
                                            _ptr(alpha), _ptr(beta), ctypes.byref(state),
                                            _ptr(out), ctypes.c_uint32(wait_limit),
                                            _stream(stream)), "lq_test_decode_step_timeout")


def lq_decode_step_host(cfg, q_host, k_host, v_host, alpha_host, beta_host, state: lq_state,
                        out_host, staging, active=None, stream=None) -> None:
    _check(_lib.lq_decode_step_host(ctypes.byref(cfg), _ptr(q_host), _ptr(k_host),
                                    _ptr(v_host), _ptr(alpha_host), _ptr(beta_host),
                                    ctypes.byref(state), _ptr(out_host), _ptr(staging),
                                    _ptr(active), _stream(stream)), "lq_decode_step_host")


def lq_decode_step_host_noalloc(cfg, q_host, k_host, v_host, alpha_host, beta_host,
                                state: lq_state, out_host, active=None, stream=None) -> None:
    """lq_decode_step_host without a staging argument, for callers that cannot
    allocate device memory: the library stages through its own fixed array of
    LQ_NOALLOC_STAGING_MAX_BYTES (shared by all calls; overlapping calls race)."""
    _check(_lib.lq_decode_step_host_noalloc(ctypes.byref(cfg), _ptr(q_host), _ptr(k_host),
                                            _ptr(v_host), _ptr(alpha_host), _ptr(beta_host),
                                            ctypes.byref(state), _ptr(out_host), _ptr(active),
                                            _stream(stream)), "lq_decode_step_host_noalloc")


def lq_window_flush(cfg, state: lq_state, mask=None, stream=None) -> None:
    _check(_lib.lq_window_flush(ctypes.byref(cfg), ctypes.byref(state), _ptr(mask),
                                _stream(stream)), "lq_window_flush")


def lq_fp32_decode_step(cfg, q, k, v, alpha, beta, S, out, stream=None) -> None:
    _check(_lib.lq_fp32_decode_step(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                    _ptr(beta), _ptr(S), _ptr(out), _stream(stream)),
           "lq_fp32_decode_step")


def lq_state_dequantize(cfg, state: lq_state, include_buffer: bool, S_out, stream=None) -> None:
    _check(_lib.lq_state_dequantize(ctypes.byref(cfg), ctypes.byref(state),
                                    1 if include_buffer else 0, _ptr(S_out), _stream(stream)),
           "lq_state_dequantize")


def lq_get_last_error(state: lq_state, stream=None) -> int:
    """Status word of the device-side checks (LQ_OK or LQ_ERR_DEVICE_BOUNDS)."""
    return _lib.lq_get_last_error(ctypes.byref(state), _stream(stream))


# ---------------------------------------------------------------------------
# The layer operators (include/leapquant_layer.h), same names
# ---------------------------------------------------------------------------

_torch = _F32 = _I32 = None
_IO = {}  # lq_dtype -> torch's


def _current():
    """(current device, current stream's handle) as torch has them; (-2, None)
    before torch has a CUDA context."""
    global _torch, _F32, _I32
    if _torch is None:
        import torch
        _F32, _I32 = torch.float32, torch.int32
        _IO.update({LQ_DTYPE_F32: torch.float32, LQ_DTYPE_BF16: torch.bfloat16})
        _torch = torch
    if not _torch.cuda.is_initialized():
        return -2, None
    dev = _torch._C._cuda_getDevice()
    return dev, _torch._C._cuda_getCurrentRawStream(dev)


def _here(x, dev: int, what: str, dtype, least: int) -> Optional[int]:
    """Address of a contiguous tensor of `dtype` (None: any) on the current
    device that holds `least` values (or an int, which is taken as it is; None)."""
    if x is None or isinstance(x, int):
        return x
    if x.get_device() != dev:
        raise ValueError(f"{what}: the tensor must be on the current CUDA device")
    if x.dtype is not dtype and dtype is not None:
        raise ValueError(f"{what}: the tensor must be {dtype}, not {x.dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{what}: the tensor must be contiguous")
    if x.numel() < least:
        raise ValueError(f"{what}: the tensor holds {x.numel()} values, the call takes {least}")
    return x.data_ptr()


def _rows(x, stride: int, dev: int, what: str, dtype, tokens: int, row: int) -> Optional[int]:
    """Address of a token-major tensor [tokens, heads, d] of `dtype` on the
    current device whose tokens lie `stride` elements apart (0: packed), each
    token's row of `row` values contiguous: a packed tensor or a slice of a fused
    projection's rows.  An int is taken as it is; `row` 0 means that the call
    does not look at it."""
    if x is None or isinstance(x, int):
        return x
    if x.get_device() != dev:
        raise ValueError(f"{what}: the tensor must be on the current CUDA device")
    if x.dtype is not dtype and dtype is not None and row:
        raise ValueError(f"{what}: the tensor must be {dtype}, not {x.dtype}")
    if stride:
        n, s = x.shape, x.stride()
        if len(s) == 3 and s[0] == stride and s[2] == 1 and s[1] == n[2] and n[0] >= tokens and \
                n[1] * s[1] >= row:
            return x.data_ptr()
    elif x.is_contiguous() and x.numel() >= tokens * row:
        return x.data_ptr()
    n, s, one = x.shape, x.stride(), 1
    for i in range(x.dim() - 1, 0, -1):
        if n[i] != 1 and s[i] != one:
            raise ValueError(f"{what}: a token's row must be contiguous")
        one *= n[i]
    if x.dim() and n[0] > 1 and one > 0 and s[0] != (stride or one):
        raise ValueError(f"{what}: tokens lie {s[0]} elements apart, "
                         f"the configuration says {stride or one}")
    held = 1 + sum((a - 1) * b for a, b in zip(n, s)) if x.numel() else 0
    need = (tokens - 1) * (stride or row) + row if tokens > 0 and row > 0 else 0
    if held < need:
        raise ValueError(f"{what}: the tensor reaches over {held} values, the call over {need}")
    return x.data_ptr()


def _on(stream, current) -> Optional[int]:
    """The handle of a call's stream: the current one by default."""
    if stream is None:
        return current
    return stream if isinstance(stream, int) else stream.cuda_stream


def make_linear_config(batch: int, num_k_heads: int, num_v_heads: int, dk: int, dv: int,
                       decay: int = LQ_DECAY_TOKEN, in_bf16: bool = False,
                       out_bf16: bool = False, q_stride: int = 0, k_stride: int = 0,
                       v_stride: int = 0) -> lq_linear_config:
    return lq_linear_config(batch, num_k_heads, num_v_heads, dk, dv, decay,
                            LQ_DTYPE_BF16 if in_bf16 else LQ_DTYPE_F32,
                            LQ_DTYPE_BF16 if out_bf16 else LQ_DTYPE_F32, q_stride, k_stride,
                            v_stride)


def lq_linear_decode_step(cfg, q, k, v, decay, S, num_slots: int, out, err, slots=None,
                          stream=None) -> None:
    """One token of S <- a S + v k^T, o = S q for every sequence, states in
    the pool S [num_slots, Hv, dv, dk] updated in place."""
    dev, now = _current()
    n, dk, hv, vrow = cfg.batch, cfg.dk, cfg.num_v_heads, cfg.num_v_heads * cfg.dv
    io, krow = _IO.get(cfg.in_dtype), cfg.num_k_heads * dk
    _check(_lib.lq_linear_decode_step(
        ctypes.byref(cfg), _rows(q, cfg.q_stride, dev, "q", io, n, krow),
        _rows(k, cfg.k_stride, dev, "k", io, n, krow),
        _rows(v, cfg.v_stride, dev, "v", io, n, vrow),
        _here(decay, dev, "decay", _F32, hv if cfg.decay else n * hv),
        _here(S, dev, "S", _F32, num_slots * vrow * dk), num_slots,
        _here(slots, dev, "slots", _I32, n),
        _here(out, dev, "out", _IO.get(cfg.out_dtype), n * vrow), _here(err, dev, "err", _I32, 1),
        _on(stream, now)), "lq_linear_decode_step")


def lq_linear_workspace_bytes(cfg, tokens: int) -> int:
    return _lib.lq_linear_workspace_bytes(ctypes.byref(cfg), tokens)


def lq_linear_prefill(cfg, q, k, v, decay, tokens: int, offsets, S, num_slots: int, out, err,
                      slots=None, fresh=None, workspace=None, stream=None) -> None:
    """The recurrence over packed prompts: sequence b owns rows
    offsets[b] .. offsets[b + 1] - 1 of `tokens`.  out may be None."""
    dev, now = _current()
    if workspace is None:
        space = 0
    elif isinstance(workspace, int):
        space = lq_linear_workspace_bytes(cfg, tokens)
    else:
        space = workspace.nbytes
    n, dk, hv, vrow = cfg.batch, cfg.dk, cfg.num_v_heads, cfg.num_v_heads * cfg.dv
    io, krow = _IO.get(cfg.in_dtype), cfg.num_k_heads * dk
    _check(_lib.lq_linear_prefill(
        ctypes.byref(cfg), _rows(q, cfg.q_stride, dev, "q", io, tokens, krow),
        _rows(k, cfg.k_stride, dev, "k", io, tokens, krow),
        _rows(v, cfg.v_stride, dev, "v", io, tokens, vrow),
        _here(decay, dev, "decay", _F32, hv if cfg.decay else tokens * hv), tokens,
        _here(offsets, dev, "offsets", _I32, n + 1),
        _here(S, dev, "S", _F32, num_slots * vrow * dk), num_slots,
        _here(slots, dev, "slots", _I32, n), _here(fresh, dev, "fresh", _I32, n),
        _here(out, dev, "out", _IO.get(cfg.out_dtype), tokens * vrow),
        _here(workspace, dev, "workspace", None, 0), space, _here(err, dev, "err", _I32, 1),
        _on(stream, now)), "lq_linear_prefill")


def lq_rotary_table(rot: int, theta: float = 10000.0, scaling: int = LQ_ROPE_NONE,
                    factor: float = 1.0, trained: float = 0.0, fast_turns: float = 32.0,
                    slow_turns: float = 1.0):
    """(table, magnitude): the rotation's table as an int64 host tensor
    [rot / 2] (the entries' 64 bits), to be moved to the device once."""
    import torch

    table = torch.empty(max(rot // 2, 1), dtype=torch.int64)
    magnitude = ctypes.c_float(1.0)
    _check(_lib.lq_rotary_table(rot, theta, scaling, factor, trained, fast_turns, slow_turns,
                                table.data_ptr(), ctypes.byref(magnitude)), "lq_rotary_table")
    return table, magnitude.value


def make_rotary_config(num_q_heads: int, num_k_heads: int, d: int, rot: int,
                       layout: int = LQ_ROPE_HALF, bf16: bool = True, magnitude: float = 1.0,
                       inverse: bool = False, q_stride: int = 0, k_stride: int = 0,
                       q_out_stride: int = 0, k_out_stride: int = 0) -> lq_rotary_config:
    return lq_rotary_config(num_q_heads, num_k_heads, d, rot, layout,
                            LQ_DTYPE_BF16 if bf16 else LQ_DTYPE_F32, 1 if inverse else 0,
                            magnitude, q_stride, k_stride, q_out_stride, k_out_stride)


def lq_rotary(cfg, tokens: int, q, k, positions, table, q_out, k_out, stream=None) -> None:
    """Rotates q and k (None without k heads) into q_out and k_out, which may
    be q and k themselves."""
    dev, now = _current()
    io, d = _IO.get(cfg.dtype), cfg.d
    qrow, krow = cfg.num_q_heads * d, cfg.num_k_heads * d
    if hasattr(table, "element_size") and table.element_size() != 8:
        raise ValueError(f"table: the tensor must hold 64-bit entries, not {table.dtype}")
    _check(_lib.lq_rotary(
        ctypes.byref(cfg), tokens, _rows(q, cfg.q_stride, dev, "q", io, tokens, qrow),
        _rows(k, cfg.k_stride, dev, "k", io, tokens, krow),
        _here(positions, dev, "positions", _I32, tokens),
        _here(table, dev, "table", None, cfg.rot // 2),
        _rows(q_out, cfg.q_out_stride, dev, "q_out", io, tokens, qrow),
        _rows(k_out, cfg.k_out_stride, dev, "k_out", io, tokens, krow), _on(stream, now)),
        "lq_rotary")


def make_norm_config(groups: int, size: int, kind: int = LQ_NORM_RMS, act: int = LQ_ACT_SILU,
                     gate_before: bool = False, shared_weight: bool = False,
                     in_bf16: bool = False, out_bf16: bool = False, eps: float = 1e-5,
                     x_stride: int = 0, gate_stride: int = 0,
                     out_stride: int = 0) -> lq_norm_config:
    return lq_norm_config(groups, size, kind, act, 1 if gate_before else 0,
                          1 if shared_weight else 0, LQ_DTYPE_BF16 if in_bf16 else LQ_DTYPE_F32,
                          LQ_DTYPE_BF16 if out_bf16 else LQ_DTYPE_F32, eps, x_stride,
                          gate_stride, out_stride)


def lq_group_norm(cfg, tokens: int, x, out, gate=None, weight=None, bias=None,
                  stream=None) -> None:
    """Normalises each token's groups; act on the result, or on the gate."""
    dev, now = _current()
    io, size = _IO.get(cfg.in_dtype), cfg.size
    row = cfg.groups * size
    _check(_lib.lq_group_norm(
        ctypes.byref(cfg), tokens, _rows(x, cfg.x_stride, dev, "x", io, tokens, row),
        _rows(gate, cfg.gate_stride, dev, "gate", io, tokens, row),
        _here(weight, dev, "weight", _F32, size if cfg.shared_weight else row),
        _here(bias, dev, "bias", _F32, row),
        _rows(out, cfg.out_stride, dev, "out", _IO.get(cfg.out_dtype), tokens, row),
        _on(stream, now)), "lq_group_norm")


def lq_get_error_word(err, stream=None) -> int:
    """Synchronizes the stream, reads and clears the error word."""
    dev, now = _current()
    return _lib.lq_get_error_word(_here(err, dev, "err", _I32, 1), _on(stream, now))


# ---------------------------------------------------------------------------
# Device memory for a state (plumbing: torch allocates, the layout decides)
# ---------------------------------------------------------------------------

class DeviceState:
    """Device buffers of one layer's stored state, allocated with torch per
    lq_state_layout.  .st is the lq_state to pass to the C calls."""

    def __init__(self, cfg: lq_config, device="cuda"):
        import torch

        self.cfg = cfg
        self.layout = L = lq_state_layout(cfg)
        u8 = torch.uint8
        self.records = torch.zeros(max(L.records_bytes, 16), dtype=u8, device=device)
        self.buf_k = torch.zeros(max(L.buf_k_bytes, 16), dtype=u8, device=device)
        self.buf_d = torch.zeros(max(L.buf_d_bytes // 4, 4), dtype=torch.float32, device=device)
        self.buf_g = torch.zeros(max(L.buf_g_bytes // 4, 4), dtype=torch.float32, device=device)
        self.buf_n = torch.zeros(max(L.buf_n_bytes // 4, 1), dtype=torch.int32, device=device)
        self.err = torch.zeros(4, dtype=torch.int32, device=device)
        self.st = lq_state(self.records.data_ptr(), self.buf_k.data_ptr(),
                           self.buf_d.data_ptr(), self.buf_g.data_ptr(),
                           self.buf_n.data_ptr(), self.err.data_ptr())

    def record_view(self):
        """[tiles, record_bytes] uint8 view of the records."""
        L, c = self.layout, self.cfg
        return self.records[:L.records_bytes].view(c.batch * c.num_v_heads, L.record_bytes)
