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
    "qw3_kv_paged_bytes", "qw3_kv_paged_append", "qw3_kv_paged_attn_workspace_bytes", "qw3_kv_paged_attn",
    "qw3_logprobs",
)

# enum qw3_type
QW3_F32 = 0
QW3_F16 = 1


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


class Qw3KvPaged(ctypes.Structure):
    """A pool of KV cache pages on a device buffer."""
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class Qw3KvBatch(ctypes.Structure):
    """A ragged batch of sequences over a paged cache."""
    _fields_ = [("starts_dev", ctypes.c_void_p), ("lens_dev", ctypes.c_void_p), ("table_dev", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("B", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32)]


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
        "qw3_kv_paged_bytes": (_I64, [_I32, _I32, _I32, _I32]),
        "qw3_kv_paged_append": (ctypes.c_int, [ctypes.POINTER(Qw3KvPaged), ctypes.POINTER(Qw3KvBatch), _I32, _P, _I32,
                                               _I64, _I32, _P, _P, _F32, _P, _I32, _P, _I64, _P, _P]),
        "qw3_kv_paged_attn_workspace_bytes": (_I64, [_I32] * 10),
        "qw3_kv_paged_attn": (ctypes.c_int, [ctypes.POINTER(Qw3KvPaged), ctypes.POINTER(Qw3KvBatch), _I32, _P, _I32,
                                             _I64, _I32, _I32, _I32, _I32, _I32, _F32, _P, _I64, _P, _I64, _P, _P]),
        "qw3_logprobs": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _P]),
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


def qw3_kv_paged_bytes(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int) -> int:
    return lib().qw3_kv_paged_bytes(n_pages, page_size, n_kv_heads, head_dim)


def qw3_kv_paged_append(cache: Qw3KvPaged, batch: Qw3KvBatch, type: int, qkv_ptr: int, M: int, qkv_stride: int,
                        n_heads: int, q_norm_ptr: int, k_norm_ptr: int, eps: float, rope_ptr: int, rope_len: int,
                        q_out_ptr: int, q_stride: int, status_ptr: int = 0, stream: int = 0) -> None:
    _check(lib().qw3_kv_paged_append(cache, batch, type, qkv_ptr or None, M, qkv_stride, n_heads, q_norm_ptr or None,
                                     k_norm_ptr or None, eps, rope_ptr or None, rope_len, q_out_ptr or None, q_stride,
                                     status_ptr or None, stream or None))


def qw3_kv_paged_attn_workspace_bytes(B: int, M: int, type: int, n_heads: int, n_kv_heads: int, head_dim: int,
                                      max_rows: int, max_len: int, window: int = 0, sinks: int = 0) -> int:
    return lib().qw3_kv_paged_attn_workspace_bytes(B, M, type, n_heads, n_kv_heads, head_dim, max_rows, max_len, window,
                                                   sinks)


def qw3_kv_paged_attn(cache: Qw3KvPaged, batch: Qw3KvBatch, type: int, q_ptr: int, M: int, q_stride: int, n_heads: int,
                      max_rows: int, max_len: int, window: int, sinks: int, scale: float, out_ptr: int, out_stride: int,
                      ws_ptr: int, ws_bytes: int, status_ptr: int = 0, stream: int = 0) -> None:
    _check(lib().qw3_kv_paged_attn(cache, batch, type, q_ptr or None, M, q_stride, n_heads, max_rows, max_len, window,
                                   sinks, scale, out_ptr or None, out_stride, ws_ptr or None, ws_bytes,
                                   status_ptr or None, stream or None))


def qw3_logprobs(logits_ptr: int, stride: int, B: int, V: int, tokens_ptr: int, T: int, top: int, logprob_ptr: int,
                 entropy_ptr: int = 0, top_id_ptr: int = 0, top_logprob_ptr: int = 0, status_ptr: int = 0,
                 stream: int = 0) -> None:
    _check(lib().qw3_logprobs(logits_ptr or None, stride, B, V, tokens_ptr or None, T, top, logprob_ptr or None,
                              entropy_ptr or None, top_id_ptr or None, top_logprob_ptr or None, status_ptr or None,
                              stream or None))


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
    if rows and width > 1 and step != 1:     # (of no rows any strides will do)
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


_kv_paged_bytes = functools.lru_cache(maxsize=256)(qw3_kv_paged_bytes)


@functools.lru_cache(maxsize=1024)
def _kv_paged_attn_workspace_bytes(device: int, *sizes: int) -> int:
    """The bytes on the current device, `device` (they go by its number of SMs)."""
    return qw3_kv_paged_attn_workspace_bytes(*sizes)


class KVCachePaged:
    """A paged f16 KV cache (qw3_kv_paged): a pool of pages that many sequences
    share. Its calls take ragged batches: rows starts[b] .. starts[b + 1] - 1 of
    the activations are the newest tokens of sequence b, which holds lens[b]
    positions with them, position p in page table[b, p // page_size] (starts int32
    [B + 1], lens int32 [B], table int32 [B, pages]; -1 where there is no page).
    Activations are f32 or f16. Every call runs on torch's current stream of the
    cache's device."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, data=None, device="cuda"):
        torch = _torch()
        # (ctypes would take a larger number modulo 2^32)
        sizes = (n_pages, page_size, n_kv_heads, head_dim)
        n = _kv_paged_bytes(*sizes) if 0 < min(sizes) and max(sizes) <= _INT32_MAX else -1
        if n < 0:
            raise Qw3Error(QW3_ERR_SHAPE, "n_pages >= 1, page_size 16, 32, 64, 128 or 256, 1 to 64 kv heads, head_dim 64 "
                                          "or 128, fewer than 2^31 rows")
        if data is None:
            if torch.device(device).type != "cuda":
                raise Qw3Error(QW3_ERR_INVALID_ARG, "device: a cache lies on a CUDA device")
            data = torch.empty((n_pages, 2, n_kv_heads, page_size, head_dim), dtype=torch.float16, device=device)
        elif data.dtype is not torch.float16 or not data.is_cuda or not data.is_contiguous() or 2 * data.numel() < n:
            raise Qw3Error(QW3_ERR_INVALID_ARG, f"data: a contiguous CUDA f16 tensor of {n // 2} values is wanted")
        self.data, self.device, self.index = data, data.device, data.get_device()
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = sizes
        self.c = Qw3KvPaged(data.data_ptr(), *sizes)

    def _batch(self, torch, starts, lens, table):
        # (written out: every call of a tensor's methods costs a short call some 0.2 of its 15 us)
        i32, index = torch.int32, self.index
        if (starts.dtype is not i32 or lens.dtype is not i32 or table.dtype is not i32 or starts.get_device() != index
                or lens.get_device() != index or table.get_device() != index or not starts.is_contiguous()
                or not lens.is_contiguous()):
            raise Qw3Error(QW3_ERR_INVALID_ARG, f"starts, lens, table: int32 tensors on cuda:{index}, starts and lens "
                                                "contiguous, are wanted")
        B = lens.numel()
        if starts.numel() != B + 1 or table.dim() != 2:
            raise Qw3Error(QW3_ERR_SHAPE, "starts holds a border more than there are sequences, table a row for each")
        rows, width = table.shape
        stride, step = table.stride()
        if rows != B or (width > 1 and step != 1) or width > _INT32_MAX or B > _INT32_MAX:
            raise Qw3Error(QW3_ERR_SHAPE, "table: a row of pages, contiguous, for each sequence is wanted")
        return Qw3KvBatch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), stride if B > 1 else width, B, width)

    def _type(self, torch, t, name):
        kind = QW3_F32 if t.dtype is torch.float32 else QW3_F16 if t.dtype is torch.float16 else -1
        if kind < 0 or t.get_device() != self.index:
            raise Qw3Error(QW3_ERR_INVALID_ARG, f"{name}: an f32 or f16 tensor on cuda:{self.index} is wanted")
        return kind

    def append(self, qkv, starts, lens, table, rope, q_norm=None, k_norm=None, eps: float = 1e-6, out=None, status=None):
        """Norm (where q_norm, k_norm: f32 [head_dim] are given), rotate and
        append the batch's rows; returns the rotated queries [M, n_heads,
        head_dim] in qkv's type (in `out` where it is given). qkv: [M, (n_heads +
        2 n_kv_heads) * head_dim], rows may be strided by multiples of 16 bytes;
        rope: f32 [positions, head_dim / 2, 2]. The queries of a row that is not
        in the cache are zero, those of rows outside the batch are not written."""
        torch = _torch()
        if _elsewhere(torch, self.index):
            with torch.cuda.device(self.index):
                return self.append(qkv, starts, lens, table, rope, q_norm, k_norm, eps, out, status)
        kind = self._type(torch, qkv, "qkv")
        M, width, stride = _rows_of(qkv, "qkv")
        hd = self.head_dim
        n_heads = width // hd - 2 * self.n_kv_heads
        if width % hd or n_heads < 1:
            raise Qw3Error(QW3_ERR_SHAPE, "qkv: rows of n_heads + 2 n_kv_heads heads are wanted")
        _on(self.index, torch.float32, "q_norm, k_norm and rope", q_norm, k_norm, rope)
        positions, half, two = rope.shape if rope.dim() == 3 else (0, 0, 0)
        if (half * 2 != hd or two != 2 or (q_norm is not None and q_norm.numel() != hd)
                or (k_norm is not None and k_norm.numel() != hd)):
            raise Qw3Error(QW3_ERR_SHAPE, "q_norm and k_norm hold head_dim values, rope [positions, head_dim / 2, 2]")
        if status is not None:
            _on(self.index, torch.int32, "status", status)
        batch = self._batch(torch, starts, lens, table)
        if out is None:
            out = qkv.new_empty((M, n_heads, hd))
        else:
            _on(self.index, qkv.dtype, "out", out)
            if out.numel() != M * n_heads * hd:
                raise Qw3Error(QW3_ERR_SHAPE, f"out: [{M}, {n_heads}, {hd}] is wanted")
        rc = lib().qw3_kv_paged_append(self.c, batch, kind, qkv.data_ptr(), M, stride, n_heads, _ptr(q_norm), _ptr(k_norm),
                                       eps, rope.data_ptr(), min(positions, _INT32_MAX), out.data_ptr(), n_heads * hd,
                                       _ptr(status), _stream_on(torch, self.index))
        if rc:
            _check(rc)
        return out

    def attention(self, q, starts, lens, table, max_rows: Optional[int] = None, max_len: Optional[int] = None,
                  window: int = 0, sinks: int = 0, scale: Optional[float] = None, out=None, workspace=None, status=None):
        """Causal attention of the batch's rows q [M, n_heads, head_dim]
        (contiguous) over the cache; returns the same shape and type. window > 0:
        a row sees its `window` newest positions and the sequence's first `sinks`.
        max_rows, max_len: upper bounds of a sequence's rows and length (M and
        what the table has pages for where they are not given); rows past
        max_rows are not written, nor are those outside the batch. They decide
        which kernels run and how the work is split: give them where they are
        known (max_rows 1 in a step of single tokens; else one sequence may have
        all the rows, and the kernel for prompts runs beside). scale:
        1 / sqrt(head_dim) where it is not given. out: where the result goes (q
        itself, or apart from it). workspace: a uint8 tensor to use in place of a
        new one."""
        torch = _torch()
        if _elsewhere(torch, self.index):
            with torch.cuda.device(self.index):
                return self.attention(q, starts, lens, table, max_rows, max_len, window, sinks, scale, out, workspace, status)
        kind = self._type(torch, q, "q")
        M, n_heads, hd = q.shape if q.dim() == 3 else (0, 0, 0)
        if hd != self.head_dim or n_heads < 1 or M > _INT32_MAX:
            raise Qw3Error(QW3_ERR_SHAPE, f"q: [M, n_heads, {self.head_dim}] is wanted")
        if not q.is_contiguous():
            raise Qw3Error(QW3_ERR_INVALID_ARG, "q: a contiguous tensor is wanted")
        if status is not None:
            _on(self.index, torch.int32, "status", status)
        if out is not None:
            _on(self.index, q.dtype, "out", out)
            if out.shape != q.shape:
                raise Qw3Error(QW3_ERR_SHAPE, "out has q's shape")
        batch = self._batch(torch, starts, lens, table)
        max_rows = M if max_rows is None else min(max_rows, M)
        max_len = batch.pages_per_seq * self.page_size if max_len is None else max_len
        if not (0 <= max_len <= _INT32_MAX and max_rows >= 0 and 0 <= window <= _INT32_MAX and 0 <= sinks <= _INT32_MAX):
            raise Qw3Error(QW3_ERR_INVALID_ARG, "a negative bound, window or sinks, or one past 31 bits")
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            need = _kv_paged_attn_workspace_bytes(self.index, batch.B, M, kind, n_heads, self.n_kv_heads, hd, max_rows,
                                                  max_len, window, sinks)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        else:
            _on(self.index, torch.uint8, "workspace", workspace)
            need = workspace.numel()
        rc = lib().qw3_kv_paged_attn(self.c, batch, kind, q.data_ptr(), M, n_heads * hd, n_heads, max_rows, max_len, window,
                                     sinks, hd ** -0.5 if scale is None else scale, out.data_ptr(), n_heads * hd,
                                     _ptr(workspace), need, _ptr(status), _stream_on(torch, self.index))
        if rc:
            _check(rc)
        return out


def logprobs(logits, tokens, top: int = 0, status=None):
    """What CUDA f32 logits [B, V] (rows may be strided) say about int32 tokens
    [B] or [B, T] (qw3_logprobs): (log probabilities of the tokens in their shape,
    entropies f32 [B], the `top` most likely tokens int32 [B, top], their log
    probabilities f32 [B, top])."""
    torch = _torch()
    B, V, stride = _rows_of(logits, "logits")
    dev = logits.get_device()
    if logits.dtype is not torch.float32 or dev < 0:
        raise Qw3Error(QW3_ERR_INVALID_ARG, "logits: a CUDA f32 tensor is wanted")
    _on(dev, torch.int32, "tokens and status", tokens, status)
    if tokens.dim() not in (1, 2) or tokens.shape[0] != B or tokens.numel() > B * _INT32_MAX:
        raise Qw3Error(QW3_ERR_SHAPE, f"tokens: [{B}] or [{B}, T] is wanted")
    if not 0 <= top <= 64:
        raise Qw3Error(QW3_ERR_SHAPE, "0 to 64 alternatives")
    if _elsewhere(torch, dev):
        with torch.cuda.device(dev):
            return logprobs(logits, tokens, top, status)
    lp = torch.empty(tokens.shape, dtype=torch.float32, device=logits.device)
    entropy = torch.empty(B, dtype=torch.float32, device=logits.device)
    top_id = torch.empty((B, top), dtype=torch.int32, device=logits.device)
    top_lp = torch.empty((B, top), dtype=torch.float32, device=logits.device)
    T = 1 if tokens.dim() == 1 else tokens.shape[1]
    rc = lib().qw3_logprobs(logits.data_ptr(), stride, B, V, tokens.data_ptr(), T, top, lp.data_ptr(), entropy.data_ptr(),
                            top_id.data_ptr(), top_lp.data_ptr(), _ptr(status), _stream_on(torch, dev))
    if rc:
        _check(rc)
    return lp, entropy, top_id, top_lp


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

    def score(self, seq: int, tokens, top: int = 0):
        """Append tokens (CUDA int32 tensor [n]) to sequence seq as
        forward_all_logits does, and return what the model makes of them: (log
        probabilities f32 [n - 1] of tokens[1:], each after the tokens before it,
        entropies f32 [n] of every row, its `top` most likely tokens int32
        [n, top] and their log probabilities f32 [n, top])."""
        torch = _torch()
        tokens = tokens.to(torch.int32).contiguous()
        logits, _ = self.forward_all_logits(seq, tokens)
        after = torch.cat((tokens[1:], tokens.new_full((1,), -1)))   # (nothing is known to follow the last one)
        lp, entropy, top_id, top_lp = logprobs(logits, after, top=top)
        return lp[:-1], entropy, top_id, top_lp

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
