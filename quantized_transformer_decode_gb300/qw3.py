"""Python binding of libqw3, the C ABI declared in include/qw3.h.

Argument marshalling only: every step of the forward pass runs in the CUDA
library. The module-level functions carry the C names and take raw pointers
(ints) like the C entry points; `Qw3Model` wraps them for torch tensors.
Importing this module does not need a GPU; loading the library does need
libqw3.so, and a missing library is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from pathlib import Path
from typing import Iterable, Optional, Sequence

import numpy as np

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libqw3.so"

QW3_OK = 0
QW3_ERR_INVALID_ARG = 1
QW3_ERR_SHAPE = 2
QW3_ERR_SEQ_POS = 3
QW3_ERR_KV_OVERFLOW = 4
QW3_ERR_NONFINITE = 5
QW3_ERR_OOM = 6
QW3_ERR_CUDA = 7
QW3_ERR_TIMEOUT = 8

QW3_FLAG_NO_GRAPH = 0x1
QW3_FLAG_NO_PDL = 0x2
QW3_FLAG_TRACE = 0x4
QW3_FLAG_PER_KERNEL = 0x8
QW3_FLAG_TEST_NO_WAIT = 0x10
QW3_FLAG_KV_F16 = 0x20
QW3_FLAG_ACT_Q8 = 0x40
QW3_FLAG_KV_Q8 = 0x80
QW3_FLAG_WEIGHTS_Q4_K = 0x100
QW3_FLAG_KV_Q4 = 0x200

# Every entry point of include/qw3.h, in declaration order.
EXPORTS = (
    "qw3_create", "qw3_destroy", "qw3_prefill", "qw3_forward_all_logits", "qw3_decode", "qw3_generate_greedy",
    "qw3_generate_sample", "qw3_reset", "qw3_truncate", "qw3_seq_len", "qw3_debug_read_kv", "qw3_debug_read_trace",
    "qw3_decode_plan", "qw3_sync", "qw3_stream", "qw3_status_string", "qw3_last_error",
    "qw3_q8_0_quantize", "qw3_q8_0_dequantize", "qw3_q8_0_gemv", "qw3_q8_0_gemv_q8act",
    "qw3_q4_k_quantize", "qw3_q4_k_dequantize", "qw3_q4_k_gemv", "qw3_q8_0_gemv_splitk_noalloc",
    "qw3_q8_0_gemm_workspace_bytes", "qw3_q8_0_gemm",
    "qw3_kv_q4_bytes", "qw3_kv_q4_append", "qw3_kv_q4_read", "qw3_kv_q4_attn_workspace_bytes", "qw3_kv_q4_attn",
    "qw3_sample",
)


class Qw3Config(ctypes.Structure):
    _fields_ = [
        ("vocab", ctypes.c_int32), ("hidden", ctypes.c_int32), ("n_layers", ctypes.c_int32),
        ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("intermediate", ctypes.c_int32), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
        ("tied_lm_head", ctypes.c_int32), ("max_seqs", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
        ("max_prefill", ctypes.c_int32), ("flags", ctypes.c_int32),
    ]


class Qw3LayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "attn_q", "attn_k", "attn_v", "attn_output", "ffn_gate", "ffn_up", "ffn_down",
        "attn_norm", "attn_q_norm", "attn_k_norm", "ffn_norm")]


class Qw3Weights(ctypes.Structure):
    _fields_ = [
        ("token_embd", ctypes.c_void_p), ("output", ctypes.c_void_p), ("output_norm", ctypes.c_void_p),
        ("layers", ctypes.POINTER(Qw3LayerWeights)), ("on_device", ctypes.c_int32),
    ]


class Qw3KvQ4(ctypes.Structure):
    """A 4-bit KV cache on a device buffer."""
    _fields_ = [("data", ctypes.c_void_p), ("slots", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class Qw3Error(RuntimeError):
    """A libqw3 call returned a non-zero status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float


def lib() -> ctypes.CDLL:
    """Load libqw3.so (built by quantized_transformer_decode_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    path = Path(os.environ.get("QW3_LIB", LIB_PATH))
    if not path.exists():
        raise RuntimeError(f"{path} is not built: run `python -m quantized_transformer_decode_gb300.build`")
    L = ctypes.CDLL(str(path))
    sig = {
        "qw3_create": (ctypes.c_int, [ctypes.POINTER(Qw3Config), ctypes.POINTER(Qw3Weights), _P, ctypes.POINTER(_P)]),
        "qw3_destroy": (ctypes.c_int, [_P]),
        "qw3_prefill": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P]),
        "qw3_forward_all_logits": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P]),
        "qw3_decode": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P]),
        "qw3_generate_greedy": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P]),
        "qw3_generate_sample": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "qw3_reset": (ctypes.c_int, [_P, _I32]),
        "qw3_truncate": (ctypes.c_int, [_P, _I32, _I32]),
        "qw3_seq_len": (ctypes.c_int, [_P, _I32, ctypes.POINTER(_I32)]),
        "qw3_debug_read_kv": (ctypes.c_int, [_P, _I32, _I32, _I32, _I32, _P, _P]),
        "qw3_debug_read_trace": (ctypes.c_int, [_P, _P, _I32, ctypes.POINTER(_I32)]),
        "qw3_decode_plan": (ctypes.c_int, [_P, _I32, ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
        "qw3_sync": (ctypes.c_int, [_P]),
        "qw3_stream": (_P, [_P]),
        "qw3_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "qw3_last_error": (ctypes.c_char_p, [_P]),
        "qw3_q8_0_quantize": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
        "qw3_q8_0_dequantize": (ctypes.c_int, [_P, _I64, _P, _P]),
        "qw3_q8_0_gemv": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _P, _P]),
        "qw3_q8_0_gemv_q8act": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _P, _P]),
        "qw3_q4_k_quantize": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
        "qw3_q4_k_dequantize": (ctypes.c_int, [_P, _I64, _P, _P]),
        "qw3_q4_k_gemv": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _P, _P]),
        "qw3_q8_0_gemv_splitk_noalloc": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _P, _P]),
        "qw3_q8_0_gemm_workspace_bytes": (_I64, [_I32, _I32, _I32]),
        "qw3_q8_0_gemm": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _P, _P, _I64, _P]),
        "qw3_kv_q4_bytes": (_I64, [_I32, _I32, _I32, _I32]),
        "qw3_kv_q4_append": (ctypes.c_int, [ctypes.POINTER(Qw3KvQ4), _P, _I32, _I64, _I32, _P, _P, _F32, _P, _P, _I32,
                                            _P, _I32, _P, _I64, _P, _P]),
        "qw3_kv_q4_read": (ctypes.c_int, [ctypes.POINTER(Qw3KvQ4), _I32, _P, _I32, _P, _I32, _P, _P, _P]),
        "qw3_kv_q4_attn_workspace_bytes": (_I64, [_I32, _I32, _I32, _I32, _I32, _I32]),
        "qw3_kv_q4_attn": (ctypes.c_int, [ctypes.POINTER(Qw3KvQ4), _P, _I64, _I32, _P, _P, _I32, _I32, _I32, _F32, _P,
                                          _I64, _P, _I64, _P, _P]),
        "qw3_sample": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(rc: int, handle=None) -> None:
    if rc != QW3_OK:
        L = lib()
        msg = (L.qw3_last_error(handle) or b"").decode(errors="replace")
        raise Qw3Error(rc, msg or L.qw3_status_string(rc).decode())


def _i32_array(vals: Optional[Sequence[int]]):
    if vals is None:
        return None
    arr = (ctypes.c_int32 * len(vals))(*[int(v) for v in vals])
    return arr


# ---------------------------------------------------------------- C names

def qw3_create(cfg: Qw3Config, weights: Qw3Weights, stream: int = 0) -> int:
    h = _P()
    rc = lib().qw3_create(ctypes.byref(cfg), ctypes.byref(weights), stream or None, ctypes.byref(h))
    _check(rc)
    return h.value


def qw3_destroy(h: int) -> None:
    _check(lib().qw3_destroy(h), h)


def qw3_prefill(h: int, seq: int, tokens_ptr: int, n: int, last_logits_ptr: int = 0, argmax_ptr: int = 0) -> None:
    _check(lib().qw3_prefill(h, seq, tokens_ptr, n, last_logits_ptr or None, argmax_ptr or None), h)


def qw3_forward_all_logits(h: int, seq: int, tokens_ptr: int, n: int, logits_ptr: int, argmax_ptr: int = 0) -> None:
    _check(lib().qw3_forward_all_logits(h, seq, tokens_ptr, n, logits_ptr or None, argmax_ptr or None), h)


def qw3_decode(h: int, B: int, seqs: Optional[Sequence[int]], tokens_ptr: int, pos: Sequence[int],
               logits_ptr: int = 0, argmax_ptr: int = 0) -> None:
    _check(lib().qw3_decode(h, B, _i32_array(seqs), tokens_ptr, _i32_array(pos), logits_ptr or None,
                            argmax_ptr or None), h)


def qw3_generate_greedy(h: int, B: int, seqs: Optional[Sequence[int]], n_steps: int, first_ptr: int,
                        out_ptr: int) -> None:
    _check(lib().qw3_generate_greedy(h, B, _i32_array(seqs), n_steps, first_ptr, out_ptr or None), h)


def qw3_generate_sample(h: int, B: int, seqs: Optional[Sequence[int]], n_steps: int, first_ptr: int,
                        temperature_ptr: int, top_k_ptr: int, top_p_ptr: int, min_p_ptr: int, u_ptr: int,
                        logits_ptr: int, out_ptr: int, prob_ptr: int = 0) -> None:
    _check(lib().qw3_generate_sample(h, B, _i32_array(seqs), n_steps, first_ptr, temperature_ptr or None,
                                     top_k_ptr or None, top_p_ptr or None, min_p_ptr or None, u_ptr or None,
                                     logits_ptr or None, out_ptr or None, prob_ptr or None), h)


def qw3_reset(h: int, seq: int) -> None:
    _check(lib().qw3_reset(h, seq), h)


def qw3_truncate(h: int, seq: int, keep_len: int) -> None:
    _check(lib().qw3_truncate(h, seq, keep_len), h)


def qw3_seq_len(h: int, seq: int) -> int:
    n = _I32()
    _check(lib().qw3_seq_len(h, seq, ctypes.byref(n)), h)
    return n.value


def qw3_debug_read_kv(h: int, layer: int, seq: int, pos0: int, n: int, k_ptr: int, v_ptr: int) -> None:
    _check(lib().qw3_debug_read_kv(h, layer, seq, pos0, n, k_ptr, v_ptr), h)


def qw3_debug_read_trace(h: int, max_records: int) -> np.ndarray:
    out = np.zeros((max_records, 8), dtype=np.uint64)
    n = _I32()
    _check(lib().qw3_debug_read_trace(h, out.ctypes.data, max_records, ctypes.byref(n)), h)
    return out[:n.value]


def qw3_decode_plan(h: int, B: int) -> tuple[bool, int]:
    """(uses the persistent step kernel, kernel launches per step)."""
    pers, lps = _I32(), _I32()
    _check(lib().qw3_decode_plan(h, B, ctypes.byref(pers), ctypes.byref(lps)), h)
    return bool(pers.value), lps.value


def qw3_sync(h: int) -> None:
    _check(lib().qw3_sync(h), h)


def qw3_stream(h: int) -> int:
    return lib().qw3_stream(h) or 0


def qw3_status_string(status: int) -> str:
    return lib().qw3_status_string(status).decode()


def qw3_last_error(h: int = 0) -> str:
    return (lib().qw3_last_error(h or None) or b"").decode(errors="replace")


def qw3_q8_0_quantize(x_ptr: int, n: int, blocks_ptr: int, status_ptr: int = 0, stream: int = 0) -> None:
    _check(lib().qw3_q8_0_quantize(x_ptr, n, blocks_ptr, status_ptr or None, stream or None))


def qw3_q8_0_dequantize(blocks_ptr: int, n: int, y_ptr: int, stream: int = 0) -> None:
    _check(lib().qw3_q8_0_dequantize(blocks_ptr, n, y_ptr, stream or None))


def qw3_q8_0_gemv(W_ptr: int, rows: int, cols: int, x_ptr: int, B: int, y_ptr: int, stream: int = 0) -> None:
    _check(lib().qw3_q8_0_gemv(W_ptr, rows, cols, x_ptr, B, y_ptr, stream or None))


def qw3_q8_0_gemv_q8act(W_ptr: int, rows: int, cols: int, x_ptr: int, B: int, y_ptr: int, stream: int = 0) -> None:
    _check(lib().qw3_q8_0_gemv_q8act(W_ptr, rows, cols, x_ptr, B, y_ptr, stream or None))


def qw3_q4_k_quantize(x_ptr: int, n: int, blocks_ptr: int, status_ptr: int = 0, stream: int = 0) -> None:
    _check(lib().qw3_q4_k_quantize(x_ptr, n, blocks_ptr, status_ptr or None, stream or None))


def qw3_q4_k_dequantize(blocks_ptr: int, n: int, y_ptr: int, stream: int = 0) -> None:
    _check(lib().qw3_q4_k_dequantize(blocks_ptr, n, y_ptr, stream or None))


def qw3_q4_k_gemv(W_ptr: int, rows: int, cols: int, x_ptr: int, B: int, y_ptr: int, stream: int = 0) -> None:
    _check(lib().qw3_q4_k_gemv(W_ptr, rows, cols, x_ptr, B, y_ptr, stream or None))


def qw3_q8_0_gemv_splitk_noalloc(W_ptr: int, rows: int, cols: int, x_ptr: int, B: int, y_ptr: int,
                                 stream: int = 0) -> None:
    _check(lib().qw3_q8_0_gemv_splitk_noalloc(W_ptr, rows, cols, x_ptr, B, y_ptr, stream or None))


def qw3_q8_0_gemm_workspace_bytes(rows: int, cols: int, M: int) -> int:
    return int(lib().qw3_q8_0_gemm_workspace_bytes(rows, cols, M))


def qw3_q8_0_gemm(W_ptr: int, rows: int, cols: int, x_ptr: int, M: int, y_ptr: int, ws_ptr: int, ws_bytes: int,
                  stream: int = 0) -> None:
    _check(lib().qw3_q8_0_gemm(W_ptr, rows, cols, x_ptr, M, y_ptr, ws_ptr or None, ws_bytes, stream or None))


def qw3_kv_q4_bytes(slots: int, capacity: int, n_kv_heads: int, head_dim: int) -> int:
    return lib().qw3_kv_q4_bytes(slots, capacity, n_kv_heads, head_dim)


def qw3_kv_q4_append(cache: Qw3KvQ4, qkv_ptr: int, M: int, qkv_stride: int, n_heads: int, q_norm_ptr: int,
                     k_norm_ptr: int, eps: float, rope_ptr: int, slots_ptr: int, slot0: int, pos_ptr: int, pos0: int,
                     q_out_ptr: int, q_stride: int, status_ptr: int = 0, stream: int = 0) -> None:
    _check(lib().qw3_kv_q4_append(cache, qkv_ptr or None, M, qkv_stride, n_heads, q_norm_ptr or None,
                                  k_norm_ptr or None, eps, rope_ptr or None, slots_ptr or None, slot0, pos_ptr or None,
                                  pos0, q_out_ptr or None, q_stride, status_ptr or None, stream or None))


def qw3_kv_q4_read(cache: Qw3KvQ4, M: int, slots_ptr: int, slot0: int, pos_ptr: int, pos0: int, k_ptr: int, v_ptr: int,
                   stream: int = 0) -> None:
    _check(lib().qw3_kv_q4_read(cache, M, slots_ptr or None, slot0, pos_ptr or None, pos0, k_ptr or None, v_ptr or None,
                                stream or None))


def qw3_kv_q4_attn_workspace_bytes(B: int, rows: int, n_heads: int, n_kv_heads: int, head_dim: int,
                                   max_len: int) -> int:
    return lib().qw3_kv_q4_attn_workspace_bytes(B, rows, n_heads, n_kv_heads, head_dim, max_len)


def qw3_kv_q4_attn(cache: Qw3KvQ4, q_ptr: int, q_stride: int, n_heads: int, slots_ptr: int, lens_ptr: int, B: int,
                   rows: int, max_len: int, scale: float, out_ptr: int, out_stride: int, ws_ptr: int, ws_bytes: int,
                   status_ptr: int = 0, stream: int = 0) -> None:
    _check(lib().qw3_kv_q4_attn(cache, q_ptr or None, q_stride, n_heads, slots_ptr or None, lens_ptr or None, B, rows,
                                max_len, scale, out_ptr or None, out_stride, ws_ptr or None, ws_bytes, status_ptr or None,
                                stream or None))


def qw3_sample(logits_ptr: int, stride: int, B: int, V: int, temperature_ptr: int, top_k_ptr: int, top_p_ptr: int,
               min_p_ptr: int, u_ptr: int, token_ptr: int, prob_ptr: int = 0, status_ptr: int = 0,
               stream: int = 0) -> None:
    _check(lib().qw3_sample(logits_ptr or None, stride, B, V, temperature_ptr or None, top_k_ptr or None,
                            top_p_ptr or None, min_p_ptr or None, u_ptr or None, token_ptr or None, prob_ptr or None,
                            status_ptr or None, stream or None))


# ---------------------------------------------------------- torch wrapper

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_ptr() -> int:
    torch = _torch()
    return torch.cuda.current_stream().cuda_stream


def q8_0_quantize(x, status=None):
    """Encode a CUDA f32 tensor (numel % 32 == 0) to Q8_0 bytes on the
    current torch stream. Returns a uint8 tensor of numel/32*34 bytes."""
    torch = _torch()
    x = x.contiguous()
    out = torch.empty(x.numel() // 32 * 34, dtype=torch.uint8, device=x.device)
    qw3_q8_0_quantize(x.data_ptr(), x.numel(), out.data_ptr(), status.data_ptr() if status is not None else 0,
                      _stream_ptr())
    return out


def q8_0_dequantize(blocks, n: int):
    torch = _torch()
    y = torch.empty(n, dtype=torch.float32, device=blocks.device)
    qw3_q8_0_dequantize(blocks.data_ptr(), n, y.data_ptr(), _stream_ptr())
    return y


def q8_0_gemv(W, rows: int, cols: int, x):
    torch = _torch()
    x = x.contiguous()
    B = x.shape[0] if x.dim() == 2 else 1
    y = torch.empty((B, rows), dtype=torch.float32, device=x.device)
    qw3_q8_0_gemv(W.data_ptr(), rows, cols, x.data_ptr(), B, y.data_ptr(), _stream_ptr())
    return y


def q8_0_gemm(W, rows: int, cols: int, x):
    """y = x . W^T for raw Q8_0 W [rows][cols] and CUDA f32 x [M][cols] on the
    tensor cores (qw3_q8_0_gemm), the workspace allocated here."""
    torch = _torch()
    x = x.contiguous()
    M = x.shape[0]
    y = torch.empty((M, rows), dtype=torch.float32, device=x.device)
    nbytes = qw3_q8_0_gemm_workspace_bytes(rows, cols, M)
    if nbytes < 0:
        raise Qw3Error(QW3_ERR_SHAPE, "cols must be a multiple of 64")
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    qw3_q8_0_gemm(W.data_ptr(), rows, cols, x.data_ptr(), M, y.data_ptr(), ws.data_ptr(), nbytes, _stream_ptr())
    return y


def q8_0_gemv_q8act(W, rows: int, cols: int, x):
    """y = W . Q8_0(x) row by row (qw3_q8_0_gemv_q8act)."""
    torch = _torch()
    x = x.contiguous()
    B = x.shape[0] if x.dim() == 2 else 1
    y = torch.empty((B, rows), dtype=torch.float32, device=x.device)
    qw3_q8_0_gemv_q8act(W.data_ptr(), rows, cols, x.data_ptr(), B, y.data_ptr(), _stream_ptr())
    return y


def q4_k_quantize(x, status=None):
    """f32 CUDA tensor (numel % 256 == 0) -> uint8 Q4_K wire bytes."""
    torch = _torch()
    x = x.contiguous()
    out = torch.empty(x.numel() // 256 * 144, dtype=torch.uint8, device=x.device)
    qw3_q4_k_quantize(x.data_ptr(), x.numel(), out.data_ptr(), status.data_ptr() if status is not None else 0,
                      _stream_ptr())
    return out


def q4_k_dequantize(blocks, n: int):
    torch = _torch()
    y = torch.empty(n, dtype=torch.float32, device=blocks.device)
    qw3_q4_k_dequantize(blocks.data_ptr(), n, y.data_ptr(), _stream_ptr())
    return y


def q4_k_gemv(W, rows: int, cols: int, x):
    torch = _torch()
    x = x.contiguous()
    B = x.shape[0] if x.dim() == 2 else 1
    y = torch.empty((B, rows), dtype=torch.float32, device=x.device)
    qw3_q4_k_gemv(W.data_ptr(), rows, cols, x.data_ptr(), B, y.data_ptr(), _stream_ptr())
    return y


_INT32_MAX = 2 ** 31 - 1


def _on(index: int, dtype, name: str, *tensors):
    """Check that each given tensor lies on CUDA device `index` as contiguous values of `dtype`."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != index or not t.is_contiguous()):
            raise Qw3Error(QW3_ERR_INVALID_ARG, f"{name}: contiguous {dtype} tensors on cuda:{index} are wanted")


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _rows_of(t, name: str):
    """(rows, width, stride) of a 2-d tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise Qw3Error(QW3_ERR_INVALID_ARG, f"{name}: a 2-d tensor with contiguous rows is wanted")
    rows, width = t.shape
    stride, step = t.stride()
    if width > 1 and step != 1:
        raise Qw3Error(QW3_ERR_INVALID_ARG, f"{name}: a 2-d tensor with contiguous rows is wanted")
    if rows > _INT32_MAX or width > _INT32_MAX:
        raise Qw3Error(QW3_ERR_SHAPE, f"{name}: more rows or columns than 31 bits count")
    return rows, width, stride if rows > 1 else max(width, stride)


def _stream_on(torch, index: int) -> int:
    """The handle of torch's current stream on device `index` (a Stream object
    around it costs a short call 2 of its 13 us)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _elsewhere(torch, index: int) -> bool:
    """Whether another device than `index` is current: a call launches on the current one."""
    return torch._C._cuda_getDevice() != index


# functions of their sizes alone, asked for in every call
_kv_q4_bytes = functools.lru_cache(maxsize=256)(qw3_kv_q4_bytes)
_kv_q4_attn_workspace_bytes = functools.lru_cache(maxsize=1024)(qw3_kv_q4_attn_workspace_bytes)


class KVCacheQ4:
    """A 4-bit KV cache of `slots` sequences (qw3_kv_q4): rows appended from
    raw q/k/v projections, read back, attended over. Every call runs on torch's
    current stream of the cache's device."""

    def __init__(self, slots: int, capacity: int, n_kv_heads: int, head_dim: int, data=None, device="cuda"):
        torch = _torch()
        # (ctypes would take a larger number modulo 2^32)
        sizes = (slots, capacity, n_kv_heads, head_dim)
        n = _kv_q4_bytes(*sizes) if 0 < min(sizes) and max(sizes) <= _INT32_MAX else -1
        if n < 0:
            raise Qw3Error(QW3_ERR_SHAPE, "slots >= 1, capacity % 32 == 0, 1 to 64 kv heads, head_dim 64 or 128")
        if data is None:
            if torch.device(device).type != "cuda":
                raise Qw3Error(QW3_ERR_INVALID_ARG, "device: a cache lies on a CUDA device")
            data = torch.empty(n, dtype=torch.uint8, device=device)
        elif data.dtype is not torch.uint8 or not data.is_cuda or not data.is_contiguous() or data.numel() < n:
            raise Qw3Error(QW3_ERR_INVALID_ARG, f"data: a contiguous CUDA uint8 tensor of {n} bytes is wanted")
        self.data, self.device, self.index = data, data.device, data.get_device()
        self.slots, self.capacity, self.n_kv_heads, self.head_dim = slots, capacity, n_kv_heads, head_dim
        self.c = Qw3KvQ4(data.data_ptr(), slots, capacity, n_kv_heads, head_dim)

    def _check_places(self, torch, M, slots, pos, slot, first):
        _on(self.index, torch.int32, "slots and pos", slots, pos)
        if not (-_INT32_MAX <= slot <= _INT32_MAX and -_INT32_MAX <= first <= _INT32_MAX and M <= _INT32_MAX):
            raise Qw3Error(QW3_ERR_INVALID_ARG, "a slot, position or row count past 31 bits")
        if (slots is not None and slots.numel() != M) or (pos is not None and pos.numel() != M):
            raise Qw3Error(QW3_ERR_SHAPE, f"slots and pos hold one place for each of {M} rows")

    def append(self, qkv, q_norm, k_norm, eps: float, rope, slots=None, pos=None, slot: int = 0, first: int = 0,
               status=None):
        """Norm, rotate and append M rows; returns the rotated queries
        [M, n_heads, head_dim]. qkv: f32 [M, (n_heads + 2 n_kv_heads) * head_dim]
        (rows may be strided); rope: f32 [capacity, head_dim / 2, 2]. Row i goes
        to (slots[i], pos[i]), int32 tensors, or to (slot, first + i). A row
        outside the cache is not cached and its queries are zero."""
        torch = _torch()
        if _elsewhere(torch, self.index):
            with torch.cuda.device(self.index):
                return self.append(qkv, q_norm, k_norm, eps, rope, slots, pos, slot, first, status)
        M, width, stride = _rows_of(qkv, "qkv")
        hd = self.head_dim
        n_heads = width // hd - 2 * self.n_kv_heads
        if qkv.dtype is not torch.float32 or qkv.get_device() != self.index or width % hd or n_heads < 1:
            raise Qw3Error(QW3_ERR_SHAPE, "qkv: f32 rows of n_heads + 2 n_kv_heads heads on the cache's device")
        _on(self.index, torch.float32, "q_norm, k_norm and rope", q_norm, k_norm, rope)
        if q_norm.numel() != hd or k_norm.numel() != hd or rope.numel() != self.capacity * hd:
            raise Qw3Error(QW3_ERR_SHAPE, "q_norm and k_norm hold head_dim values, rope capacity * head_dim")
        if status is not None:
            _on(self.index, torch.int32, "status", status)
        self._check_places(torch, M, slots, pos, slot, first)
        q = torch.empty((M, n_heads, hd), dtype=torch.float32, device=self.device)
        rc = lib().qw3_kv_q4_append(self.c, qkv.data_ptr(), M, stride, n_heads, q_norm.data_ptr(), k_norm.data_ptr(),
                                    eps, rope.data_ptr(), _ptr(slots), slot, _ptr(pos), first, q.data_ptr(),
                                    n_heads * hd, _ptr(status), _stream_on(torch, self.index))
        if rc:
            _check(rc)
        return q

    def read(self, slots=None, pos=None, slot: int = 0, first: int = 0, n: Optional[int] = None):
        """Rows back as f32: (k, v), each [M, n_kv_heads, head_dim]; the places
        as in append, M from slots or pos, else n. Rows outside the cache are
        zero."""
        torch = _torch()
        if _elsewhere(torch, self.index):
            with torch.cuda.device(self.index):
                return self.read(slots, pos, slot, first, n)
        M = n if n is not None else slots.numel() if slots is not None else pos.numel() if pos is not None else -1
        if M < 0:
            raise Qw3Error(QW3_ERR_INVALID_ARG, "read needs slots, pos or n")
        self._check_places(torch, M, slots, pos, slot, first)
        shape = (M, self.n_kv_heads, self.head_dim)
        k = torch.empty(shape, dtype=torch.float32, device=self.device)
        v = torch.empty(shape, dtype=torch.float32, device=self.device)
        rc = lib().qw3_kv_q4_read(self.c, M, _ptr(slots), slot, _ptr(pos), first, k.data_ptr(), v.data_ptr(),
                                  _stream_on(torch, self.index))
        if rc:
            _check(rc)
        return k, v

    def attention(self, q, lens, rows: int = 1, slots=None, max_len: Optional[int] = None,
                  scale: Optional[float] = None, out=None, workspace=None, status=None):
        """Attention of q [B * rows, n_heads, head_dim] (f32, contiguous) over
        the first lens[b] positions (int32 [B]) of slot slots[b] (int32 [B],
        else slot b); returns the same shape. max_len: an upper bound of lens
        (the capacity where it is not given). scale: 1 / sqrt(head_dim) where it
        is not given. out: where the result goes (q itself, or apart from it).
        workspace: a uint8 tensor to use in place of a new one."""
        torch = _torch()
        if _elsewhere(torch, self.index):
            with torch.cuda.device(self.index):
                return self.attention(q, lens, rows, slots, max_len, scale, out, workspace, status)
        B, hd, n_heads = lens.numel(), self.head_dim, q.shape[1] if q.dim() == 3 else 0
        _on(self.index, torch.float32, "q and out", q, out)
        _on(self.index, torch.int32, "lens, slots and status", lens, slots, status)
        if n_heads < 1 or q.shape[0] != B * rows or q.shape[2] != hd:
            raise Qw3Error(QW3_ERR_SHAPE, f"q: [{B * rows}, n_heads, {hd}] is wanted")
        if (slots is not None and slots.numel() != B) or (out is not None and out.shape != q.shape):
            raise Qw3Error(QW3_ERR_SHAPE, "slots holds one slot per sequence, out has q's shape")
        if slots is None and B > self.slots:
            raise Qw3Error(QW3_ERR_SHAPE, "more sequences than slots")
        max_len = self.capacity if max_len is None else max_len
        if not 0 <= max_len <= self.capacity:
            raise Qw3Error(QW3_ERR_KV_OVERFLOW if max_len > 0 else QW3_ERR_INVALID_ARG, "max_len past the cache's capacity")
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            need = _kv_q4_attn_workspace_bytes(B, rows, n_heads, self.n_kv_heads, hd, max_len)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        else:
            _on(self.index, torch.uint8, "workspace", workspace)
            need = workspace.numel()
        rc = lib().qw3_kv_q4_attn(self.c, q.data_ptr(), n_heads * hd, n_heads, _ptr(slots), lens.data_ptr(), B, rows,
                                  max_len, hd ** -0.5 if scale is None else scale, out.data_ptr(), n_heads * hd,
                                  _ptr(workspace), need, _ptr(status), _stream_on(torch, self.index))
        if rc:
            _check(rc)
        return out


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, status=None):
    """One token per row of CUDA f32 logits [B, V] (rows may be strided) from
    uniform numbers u [B] (qw3_sample): (tokens int32 [B], probabilities f32
    [B]). temperature, top_p, min_p: f32 [B]; top_k: int32 [B]; each may be
    left out."""
    torch = _torch()
    B, V, stride = _rows_of(logits, "logits")
    dev = logits.get_device()
    if logits.dtype is not torch.float32 or dev < 0:
        raise Qw3Error(QW3_ERR_INVALID_ARG, "logits: a CUDA f32 tensor is wanted")
    _on(dev, torch.float32, "u, temperature, top_p and min_p", u, temperature, top_p, min_p)
    _on(dev, torch.int32, "top_k and status", top_k, status)
    for t in (u, temperature, top_k, top_p, min_p):
        if t is not None and t.numel() != B:
            raise Qw3Error(QW3_ERR_SHAPE, f"one setting and one number for each of {B} rows are wanted")
    if _elsewhere(torch, dev):
        with torch.cuda.device(dev):
            return sample(logits, u, temperature, top_k, top_p, min_p, status)
    token = torch.empty(B, dtype=torch.int32, device=logits.device)
    prob = torch.empty(B, dtype=torch.float32, device=logits.device)
    rc = lib().qw3_sample(logits.data_ptr(), stride, B, V, _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
                          u.data_ptr(), token.data_ptr(), prob.data_ptr(), _ptr(status), _stream_on(torch, dev))
    if rc:
        _check(rc)
    return token, prob


class _Ordered:
    """Orders the model's stream after torch's current stream on entry and
    torch's current stream after the model's stream on exit, so tensors that
    torch wrote are ready and temporaries freed by torch are not reused while
    the library still reads them."""

    def __init__(self, model: "Qw3Model"):
        self.m = model

    def __enter__(self):
        torch = _torch()
        self.cur = torch.cuda.current_stream()
        self.m.stream.wait_stream(self.cur)
        return self

    def __exit__(self, *exc):
        self.cur.wait_stream(self.m.stream)
        return False


class Qw3Model:
    """A libqw3 model on its own torch-owned CUDA stream.

    Build it from f32 weights (quantised on the device by the library's Q8_0
    encoder) or from Q8_0 bytes in GGUF layout.
    """

    def __init__(self, shape, tensors_dev: dict, *, max_seqs: int = 1, max_seq_len: int = 1024,
                 max_prefill: int = 512, flags: int = 0):
        torch = _torch()
        self.shape = shape
        self.stream = torch.cuda.Stream()
        self.max_seqs, self.max_seq_len, self.max_prefill = max_seqs, max_seq_len, max_prefill
        cfg = Qw3Config(vocab=shape.vocab, hidden=shape.hidden, n_layers=shape.n_layers, n_heads=shape.n_heads,
                        n_kv_heads=shape.n_kv_heads, head_dim=shape.head_dim, intermediate=shape.intermediate,
                        rms_eps=shape.rms_eps, rope_theta=shape.rope_theta, tied_lm_head=1 if shape.tied else 0,
                        max_seqs=max_seqs, max_seq_len=max_seq_len, max_prefill=max_prefill, flags=flags)
        layers = (Qw3LayerWeights * shape.n_layers)()
        names = ("attn_q", "attn_k", "attn_v", "attn_output", "ffn_gate", "ffn_up", "ffn_down",
                 "attn_norm", "attn_q_norm", "attn_k_norm", "ffn_norm")
        for i in range(shape.n_layers):
            for nm in names:
                setattr(layers[i], nm, tensors_dev[f"blk.{i}.{nm}"].data_ptr())
        w = Qw3Weights(token_embd=tensors_dev["token_embd"].data_ptr(),
                       output=tensors_dev["output"].data_ptr() if not shape.tied else None,
                       output_norm=tensors_dev["output_norm"].data_ptr(), layers=layers, on_device=1)
        # the weights were written on torch's current stream
        self.stream.wait_stream(torch.cuda.current_stream())
        self.h = qw3_create(cfg, w, self.stream.cuda_stream)
        self.flags = flags

    @classmethod
    def from_f32(cls, shape, weights: Iterable, device: str = "cuda", **kw) -> "Qw3Model":
        """weights: iterable of (name, kind, f32 numpy array) in any order;
        linear tensors are quantised on the device with qw3_q8_0_quantize, or
        qw3_q4_k_quantize when flags hold QW3_FLAG_WEIGHTS_Q4_K."""
        torch = _torch()
        tensors = {}
        status = torch.zeros(1, dtype=torch.int32, device=device)
        enc = q4_k_quantize if kw.get("flags", 0) & QW3_FLAG_WEIGHTS_Q4_K else q8_0_quantize
        for name, kind, arr in weights:
            t = torch.from_numpy(np.ascontiguousarray(arr, dtype=np.float32)).to(device)
            tensors[name] = enc(t.reshape(-1), status) if kind == "linear" else t
            del t
        if int(status.item()) != 0:
            raise Qw3Error(int(status.item()), "non-finite weight values")
        m = cls(shape, tensors, **kw)
        del tensors
        return m

    @classmethod
    def from_q8_0(cls, shape, tensors_host: dict, device: str = "cuda", **kw) -> "Qw3Model":
        """tensors_host: GGUF name -> Q8_0 wire bytes (linear) or f32 (norm)."""
        torch = _torch()
        dev = {k: torch.from_numpy(np.ascontiguousarray(v)).to(device) for k, v in tensors_host.items()}
        return cls(shape, dev, **kw)

    # -- calls ---------------------------------------------------------------

    def prefill(self, seq: int, tokens, want_logits: bool = True):
        """Append tokens (CUDA int32 tensor) to sequence seq; return
        (last-row logits or None, argmax int32 tensor [1])."""
        torch = _torch()
        tokens = tokens.to(torch.int32).contiguous()
        logits = torch.empty(self.shape.vocab, dtype=torch.float32, device=tokens.device) if want_logits else None
        am = torch.empty(1, dtype=torch.int32, device=tokens.device)
        with _Ordered(self):
            qw3_prefill(self.h, seq, tokens.data_ptr(), tokens.numel(),
                        logits.data_ptr() if logits is not None else 0, am.data_ptr())
        return logits, am

    def forward_all_logits(self, seq: int, tokens):
        """Append tokens (CUDA int32 tensor [n]) to sequence seq; return
        (logits [n, vocab], argmax int32 [n]) of every appended row."""
        torch = _torch()
        tokens = tokens.to(torch.int32).contiguous()
        n = tokens.numel()
        logits = torch.empty((n, self.shape.vocab), dtype=torch.float32, device=tokens.device)
        am = torch.empty(n, dtype=torch.int32, device=tokens.device)
        with _Ordered(self):
            qw3_forward_all_logits(self.h, seq, tokens.data_ptr(), n, logits.data_ptr(), am.data_ptr())
        return logits, am

    def decode(self, tokens, pos: Sequence[int], seqs: Optional[Sequence[int]] = None, want_logits: bool = True):
        """One decode step for B = len(pos) sequences; tokens CUDA int32 [B]."""
        torch = _torch()
        B = len(pos)
        tokens = tokens.to(torch.int32).contiguous()
        logits = torch.empty((B, self.shape.vocab), dtype=torch.float32,
                             device=tokens.device) if want_logits else None
        am = torch.empty(B, dtype=torch.int32, device=tokens.device)
        with _Ordered(self):
            qw3_decode(self.h, B, seqs, tokens.data_ptr(), pos, logits.data_ptr() if logits is not None else 0,
                       am.data_ptr())
        return logits, am

    def generate_greedy(self, first_tokens, n_steps: int, seqs: Optional[Sequence[int]] = None, out=None):
        torch = _torch()
        first_tokens = first_tokens.to(torch.int32).contiguous()
        B = first_tokens.numel()
        if out is None:
            out = torch.empty((n_steps, B), dtype=torch.int32, device=first_tokens.device)
        with _Ordered(self):
            qw3_generate_greedy(self.h, B, seqs, n_steps, first_tokens.data_ptr(), out.data_ptr())
        return out

    def generate_sample(self, first_tokens, n_steps: int, u, temperature=None, top_k=None, top_p=None, min_p=None,
                        seqs: Optional[Sequence[int]] = None):
        """n_steps sampled steps (qw3_generate_sample) from tensors on the model's
        device: first_tokens [B], u f32 [n_steps, B] in [0, 1), the settings [B]
        each (f32; top_k int32) or left out. Returns (tokens int32 [n_steps, B],
        probabilities f32 [n_steps, B])."""
        torch = _torch()
        first_tokens = first_tokens.to(torch.int32).contiguous()
        B, dev = first_tokens.numel(), self.stream.device.index
        _on(dev, torch.int32, "first_tokens", first_tokens)
        _on(dev, torch.float32, "u, temperature, top_p and min_p", u, temperature, top_p, min_p)
        _on(dev, torch.int32, "top_k", top_k)
        if u.numel() != n_steps * B or any(t is not None and t.numel() != B for t in (temperature, top_k, top_p, min_p)):
            raise Qw3Error(QW3_ERR_SHAPE, "u holds n_steps * B numbers, a setting B")
        if seqs is not None and len(seqs) != B:
            raise Qw3Error(QW3_ERR_SHAPE, "seqs names one sequence for each first token")
        logits = torch.empty((B, self.shape.vocab), dtype=torch.float32, device=first_tokens.device)
        out = torch.empty((n_steps, B), dtype=torch.int32, device=first_tokens.device)
        prob = torch.empty((n_steps, B), dtype=torch.float32, device=first_tokens.device)
        with _Ordered(self):
            qw3_generate_sample(self.h, B, seqs, n_steps, first_tokens.data_ptr(), _ptr(temperature), _ptr(top_k),
                                _ptr(top_p), _ptr(min_p), u.data_ptr(), logits.data_ptr(), out.data_ptr(),
                                prob.data_ptr())
        return out, prob

    def reset(self, seq: int) -> None:
        qw3_reset(self.h, seq)

    def truncate(self, seq: int, keep_len: int) -> None:
        qw3_truncate(self.h, seq, keep_len)

    def seq_len(self, seq: int) -> int:
        return qw3_seq_len(self.h, seq)

    def read_kv(self, layer: int, seq: int, pos0: int, n: int):
        torch = _torch()
        s = self.shape
        k = torch.empty((n, s.n_kv_heads, s.head_dim), dtype=torch.float32, device="cuda")
        v = torch.empty_like(k)
        with _Ordered(self):
            qw3_debug_read_kv(self.h, layer, seq, pos0, n, k.data_ptr(), v.data_ptr())
        return k, v

    def read_trace(self, max_records: int = 4096) -> np.ndarray:
        return qw3_debug_read_trace(self.h, max_records)

    def decode_plan(self, B: int = 1) -> tuple[bool, int]:
        return qw3_decode_plan(self.h, B)

    def sync(self) -> None:
        qw3_sync(self.h)

    def close(self) -> None:
        if getattr(self, "h", None):
            qw3_destroy(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
        return False

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
