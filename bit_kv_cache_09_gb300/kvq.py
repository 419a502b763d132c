"""ctypes binding of libkvq (the C ABI in include/kvq.h).

Argument marshalling only: every step of the quantized-KV path runs in the CUDA
kernels of ``libkvq.so``. Each function keeps the C name and raises ``KVQError``
on a non-OK status. Pointers are plain integers (``tensor.data_ptr()``) and the
stream is a ``cudaStream_t`` value (``torch.cuda.current_stream().cuda_stream``).
Loading fails loudly when the library has not been built.
"""

from __future__ import annotations

import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvq.so")

KVQ_OK = 0
STATUS_NAMES = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED", 3: "KVQ_ERR_CAPACITY",
                4: "KVQ_ERR_WORKSPACE", 5: "KVQ_ERR_CUDA"}
BUFFER_NAMES = ("k_codes", "k_meta", "k_resid", "v_codes", "v_meta")
DECODE_AUTO, DECODE_SIMT, DECODE_MMA = 0, 1, 2
DECODE_EARLY_PREFETCH = 1  # flag bits of kvq_decode_attention_ex / kvq_decode_step_ex
DECODE_ZERO_WAIT_LIMIT = 2
DECODE_ERR_WAIT_TIMEOUT = 1  # bit of the decode error word
EXPORTED = ("kvq_buffer_sizes", "kvq_quantize_append", "kvq_dequantize", "kvq_decode_workspace_size",
            "kvq_decode_attention", "kvq_decode_attention_impl", "kvq_decode_num_splits", "kvq_status_string",
            "kvq_version", "kvq_decode_attention_noalloc", "kvq_decode_step", "kvq_decode_attention_ex",
            "kvq_decode_step_ex", "kvq_decode_error", "kvq_decode_noalloc_error", "kvq_paged_buffer_sizes",
            "kvq_paged_step_tables", "kvq_paged_append", "kvq_paged_dequantize", "kvq_paged_workspace_size",
            "kvq_paged_decode_attention", "kvq_prompt_workspace_size", "kvq_prompt_attention")
PAGED_FORMATS = {"int8": 0, "e4m3": 1}  # kvq_paged_config.format
F16, BF16 = 0, 1  # 16-bit types of the paged cache and of the prompt attention
PAGED_ERR_NEW, PAGED_ERR_LENGTH, PAGED_ERR_BLOCKS, PAGED_ERR_STATE = 1, 2, 4, 8  # bits of step.status[0]
PAGED_ERR_ROWS, PAGED_ERR_TABLE = 16, 32
PAGED_ZERO_REST, PAGED_EARLY_TABLES, PAGED_ZERO_WAIT_LIMIT = 1, 2, 4  # flag bits of kvq_paged_decode_attention
PROMPT_ZERO_REST, PROMPT_ZERO_WAIT_LIMIT = 1, 2  # flag bits of kvq_prompt_args
PAGED_ERR_NAMES = {1: "new_tokens below -1 or more than max_new in all", 2: "a request outgrows max_blocks",
                   4: "not enough free blocks", 8: "lengths or free count out of range",
                   16: "fewer key/value rows than the step's new tokens", 32: "a block number outside the pool"}


class KVQError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({message})")
        self.status = status


class KVQDeviceError(RuntimeError):
    """A decode launch reported a device-side error in its workspace error word."""

    def __init__(self, word: int):
        names = [n for bit, n in ((DECODE_ERR_WAIT_TIMEOUT, "a wait for staged cache tiles timed out"),) if word & bit]
        super().__init__(f"decode error word 0x{word:x}: {'; '.join(names) or 'unknown bits'}")
        self.word = word


class KVQStepError(RuntimeError):
    """A step of the paged cache recorded an error (bits PAGED_ERR_* of its status word)."""

    def __init__(self, bits: int):
        names = [n for bit, n in PAGED_ERR_NAMES.items() if bits & bit]
        super().__init__(f"step status 0x{bits:x}: {'; '.join(names) or 'unknown bits'}")
        self.bits = bits


class kvq_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "batch", "n_kv_heads", "gqa_ratio", "d_head",
                                               "max_seq_len", "bits", "k_group", "v_group", "residual_len",
                                               "v_bits", "symmetric", "k_outliers")]


class kvq_buffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in BUFFER_NAMES]


class kvq_paged_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "n_kv_heads", "gqa_ratio", "d_head", "n_blocks",
                                               "block_tokens", "n_requests", "max_blocks", "max_new", "format",
                                               "dtype")]


class kvq_paged_buffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "scales", "tails")]


class kvq_paged_state(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("lens", "block_table", "free_list", "free_count")]


class kvq_paged_step(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("lens", "free_count", "q_start", "positions", "slots", "units",
                                               "tile_start", "status")]


class kvq_prompt_args(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("n_kv_heads", "gqa_ratio", "d_head", "dtype", "n_seqs", "causal", "flags")]
                + [(n, ctypes.c_int64) for n in ("n_q", "n_kv")] + [(n, ctypes.c_void_p) for n in ("q", "k", "v")]
                + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "out_stride")]
                + [(n, ctypes.c_void_p) for n in ("q_start", "kv_start")] + [("softmax_scale", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("out", "lse")])


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkvq.so; raises if it is missing (build it with bit_kv_cache_09_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libkvq.so not found at {path}: run `python -m bit_kv_cache_09_gb300.build` "
                               "(the quantized-KV path has no fallback)")
        L = ctypes.CDLL(path)
        cfgp, bufp, vp = ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_buffers), ctypes.c_void_p
        L.kvq_buffer_sizes.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
        L.kvq_buffer_sizes.restype = ctypes.c_int
        L.kvq_quantize_append.argtypes = [cfgp, bufp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, vp, vp, vp]
        L.kvq_quantize_append.restype = ctypes.c_int
        L.kvq_dequantize.argtypes = [cfgp, bufp, ctypes.c_int32, ctypes.c_int64, vp, vp, vp]
        L.kvq_dequantize.restype = ctypes.c_int
        L.kvq_decode_workspace_size.argtypes = [cfgp, ctypes.c_int64]
        L.kvq_decode_workspace_size.restype = ctypes.c_size_t
        L.kvq_decode_attention.argtypes = [cfgp, bufp, ctypes.c_int32, ctypes.c_int64, vp, ctypes.c_float, vp, vp,
                                           ctypes.c_size_t, vp]
        L.kvq_decode_attention.restype = ctypes.c_int
        L.kvq_decode_attention_impl.argtypes = L.kvq_decode_attention.argtypes + [ctypes.c_int]
        L.kvq_decode_attention_impl.restype = ctypes.c_int
        L.kvq_decode_attention_noalloc.argtypes = [cfgp, bufp, ctypes.c_int32, ctypes.c_int64, vp, ctypes.c_float,
                                                   vp, vp]
        L.kvq_decode_attention_noalloc.restype = ctypes.c_int
        L.kvq_decode_step.argtypes = [cfgp, bufp, ctypes.c_int32, ctypes.c_int64, vp, vp, vp, ctypes.c_float, vp, vp,
                                      ctypes.c_size_t, vp]
        L.kvq_decode_step.restype = ctypes.c_int
        L.kvq_decode_attention_ex.argtypes = L.kvq_decode_attention.argtypes + [ctypes.c_uint32]
        L.kvq_decode_attention_ex.restype = ctypes.c_int
        L.kvq_decode_step_ex.argtypes = L.kvq_decode_step.argtypes + [ctypes.c_uint32]
        L.kvq_decode_step_ex.restype = ctypes.c_int
        L.kvq_decode_error.argtypes = [vp, ctypes.c_size_t, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.kvq_decode_error.restype = ctypes.c_int
        L.kvq_decode_noalloc_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        L.kvq_decode_noalloc_error.restype = ctypes.c_int
        L.kvq_decode_num_splits.argtypes = [cfgp, ctypes.c_int64]
        L.kvq_decode_num_splits.restype = ctypes.c_int32
        pcfg, pbuf, pstep = (ctypes.POINTER(t) for t in (kvq_paged_config, kvq_paged_buffers, kvq_paged_step))
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        L.kvq_paged_buffer_sizes.argtypes = [pcfg, ctypes.POINTER(ctypes.c_size_t)]
        L.kvq_paged_buffer_sizes.restype = ctypes.c_int
        L.kvq_paged_step_tables.argtypes = [pcfg, ctypes.POINTER(kvq_paged_state), vp, pstep, i32, vp]
        L.kvq_paged_step_tables.restype = ctypes.c_int
        L.kvq_paged_append.argtypes = [pcfg, pbuf, vp, pstep, i32, i64, vp, i64, vp, i64, vp]
        L.kvq_paged_append.restype = ctypes.c_int
        L.kvq_paged_dequantize.argtypes = [pcfg, pbuf, i32, i64, vp, vp, vp, vp]
        L.kvq_paged_dequantize.restype = ctypes.c_int
        L.kvq_paged_workspace_size.argtypes = [pcfg]
        L.kvq_paged_workspace_size.restype = ctypes.c_size_t
        L.kvq_paged_decode_attention.argtypes = [pcfg, pbuf, vp, pstep, i32, vp, i64, ctypes.c_float, vp,
                                                 ctypes.c_uint32,
                                                 vp, ctypes.c_size_t, vp]
        L.kvq_paged_decode_attention.restype = ctypes.c_int
        L.kvq_prompt_workspace_size.argtypes = []
        L.kvq_prompt_workspace_size.restype = ctypes.c_size_t
        L.kvq_prompt_attention.argtypes = [ctypes.POINTER(kvq_prompt_args), vp, ctypes.c_size_t, vp]
        L.kvq_prompt_attention.restype = ctypes.c_int
        L.kvq_status_string.argtypes = [ctypes.c_int]
        L.kvq_status_string.restype = ctypes.c_char_p
        L.kvq_version.argtypes = []
        L.kvq_version.restype = ctypes.c_char_p
        _lib = L
        return L


def _check(fn: str, status: int) -> None:
    if status != KVQ_OK:
        raise KVQError(fn, status, kvq_status_string(status))


def make_config(*, n_layers, batch, n_kv_heads, gqa_ratio, d_head, max_seq_len, bits, k_group, v_group,
                residual_len, v_bits=0, symmetric=0, k_outliers=0) -> kvq_config:
    return kvq_config(n_layers, batch, n_kv_heads, gqa_ratio, d_head, max_seq_len, bits, k_group, v_group,
                      residual_len, v_bits, int(symmetric), int(k_outliers))


def make_buffers(ptrs) -> kvq_buffers:
    """ptrs: five device addresses (ints) in the order k_codes, k_meta, k_resid, v_codes, v_meta."""
    return kvq_buffers(*[ctypes.c_void_p(int(p)) for p in ptrs])


def kvq_status_string(status: int) -> str:
    return load().kvq_status_string(int(status)).decode()


def kvq_version() -> str:
    return load().kvq_version().decode()


def kvq_buffer_sizes(cfg: kvq_config) -> list[int]:
    out = (ctypes.c_size_t * 5)()
    _check("kvq_buffer_sizes", load().kvq_buffer_sizes(ctypes.byref(cfg), out))
    return [int(v) for v in out]


def kvq_quantize_append(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, n_new: int, k_f16: int,
                        v_f16: int, stream: int = 0) -> None:
    _check("kvq_quantize_append", load().kvq_quantize_append(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur,
                                                             n_new, k_f16, v_f16, stream))


def kvq_dequantize(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, k_out: int, v_out: int,
                   stream: int = 0) -> None:
    _check("kvq_dequantize", load().kvq_dequantize(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur, k_out,
                                                   v_out, stream))


def kvq_decode_workspace_size(cfg: kvq_config, s_cur: int) -> int:
    return int(load().kvq_decode_workspace_size(ctypes.byref(cfg), s_cur))


def kvq_decode_num_splits(cfg: kvq_config, s_cur: int) -> int:
    return int(load().kvq_decode_num_splits(ctypes.byref(cfg), s_cur))


def kvq_decode_attention(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, q_f16: int,
                         softmax_scale: float, out: int, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check("kvq_decode_attention", load().kvq_decode_attention(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur,
                                                               q_f16, softmax_scale, out, ws, ws_bytes, stream))


def kvq_decode_attention_impl(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, q_f16: int,
                              softmax_scale: float, out: int, ws: int, ws_bytes: int, stream: int = 0,
                              impl: int = DECODE_AUTO) -> None:
    _check("kvq_decode_attention_impl",
           load().kvq_decode_attention_impl(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur, q_f16, softmax_scale,
                                            out, ws, ws_bytes, stream, impl))


def kvq_decode_step(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, k_f16: int, v_f16: int, q_f16: int,
                    softmax_scale: float, out: int, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check("kvq_decode_step", load().kvq_decode_step(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur, k_f16, v_f16,
                                                     q_f16, softmax_scale, out, ws, ws_bytes, stream))


def kvq_decode_attention_ex(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, q_f16: int,
                            softmax_scale: float, out: int, ws: int, ws_bytes: int, stream: int = 0,
                            flags: int = 0) -> None:
    _check("kvq_decode_attention_ex",
           load().kvq_decode_attention_ex(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur, q_f16, softmax_scale,
                                          out, ws, ws_bytes, stream, flags))


def kvq_decode_step_ex(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, k_f16: int, v_f16: int,
                       q_f16: int, softmax_scale: float, out: int, ws: int, ws_bytes: int, stream: int = 0,
                       flags: int = 0) -> None:
    _check("kvq_decode_step_ex", load().kvq_decode_step_ex(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur, k_f16,
                                                           v_f16, q_f16, softmax_scale, out, ws, ws_bytes, stream,
                                                           flags))


def kvq_decode_attention_noalloc(cfg: kvq_config, bufs: kvq_buffers, layer: int, s_cur: int, q_f16: int,
                                 softmax_scale: float, out: int, stream: int = 0) -> None:
    """Decode attention with the library's static 16 MiB device scratch instead of a
    caller workspace (for callers that cannot allocate; calls must not overlap)."""
    _check("kvq_decode_attention_noalloc",
           load().kvq_decode_attention_noalloc(ctypes.byref(cfg), ctypes.byref(bufs), layer, s_cur, q_f16,
                                               softmax_scale, out, stream))


def kvq_decode_error(ws: int, ws_bytes: int, stream: int = 0) -> int:
    """The decode error word of workspace `ws` (synchronizes `stream`, then clears it)."""
    word = ctypes.c_uint32(0)
    _check("kvq_decode_error", load().kvq_decode_error(ws, ws_bytes, stream, ctypes.byref(word)))
    return int(word.value)


def kvq_decode_noalloc_error(stream: int = 0) -> int:
    """The error word of the last kvq_decode_attention_noalloc call on the current device."""
    word = ctypes.c_uint32(0)
    _check("kvq_decode_noalloc_error", load().kvq_decode_noalloc_error(stream, ctypes.byref(word)))
    return int(word.value)


def make_paged_config(*, n_layers, n_kv_heads, gqa_ratio, d_head, n_blocks, block_tokens, n_requests, max_blocks,
                      max_new, fmt, dtype) -> kvq_paged_config:
    """fmt: a key of PAGED_FORMATS (or its number); dtype: F16 or BF16."""
    return kvq_paged_config(n_layers, n_kv_heads, gqa_ratio, d_head, n_blocks, block_tokens, n_requests, max_blocks,
                            max_new, PAGED_FORMATS.get(fmt, fmt), dtype)


def kvq_paged_buffer_sizes(cfg: kvq_paged_config) -> list[int]:
    out = (ctypes.c_size_t * 3)()
    _check("kvq_paged_buffer_sizes", load().kvq_paged_buffer_sizes(ctypes.byref(cfg), out))
    return [int(v) for v in out]


def kvq_paged_workspace_size(cfg: kvq_paged_config) -> int:
    return int(load().kvq_paged_workspace_size(ctypes.byref(cfg)))


def kvq_paged_step_tables(cfg: kvq_paged_config, state: kvq_paged_state, new_tokens: int, step: kvq_paged_step,
                          commit: int = 1, stream: int = 0) -> None:
    _check("kvq_paged_step_tables", load().kvq_paged_step_tables(ctypes.byref(cfg), ctypes.byref(state), new_tokens,
                                                                 ctypes.byref(step), commit, stream))


def kvq_paged_append(cfg: kvq_paged_config, bufs: kvq_paged_buffers, block_table: int, step: kvq_paged_step,
                     layer: int, n_rows: int, k: int, k_stride: int, v: int, v_stride: int, stream: int = 0) -> None:
    _check("kvq_paged_append", load().kvq_paged_append(ctypes.byref(cfg), ctypes.byref(bufs), block_table,
                                                       ctypes.byref(step), layer, n_rows, k, k_stride, v, v_stride,
                                                       stream))


def kvq_paged_dequantize(cfg: kvq_paged_config, bufs: kvq_paged_buffers, layer: int, n: int, slots: int, k_out: int,
                         v_out: int, stream: int = 0) -> None:
    _check("kvq_paged_dequantize", load().kvq_paged_dequantize(ctypes.byref(cfg), ctypes.byref(bufs), layer, n, slots,
                                                               k_out, v_out, stream))


def kvq_paged_decode_attention(cfg: kvq_paged_config, bufs: kvq_paged_buffers, block_table: int, step: kvq_paged_step,
                               layer: int, q: int, q_stride: int, softmax_scale: float, out: int, flags: int,
                               ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check("kvq_paged_decode_attention",
           load().kvq_paged_decode_attention(ctypes.byref(cfg), ctypes.byref(bufs), block_table, ctypes.byref(step),
                                             layer, q, q_stride, softmax_scale, out, flags, ws, ws_bytes,
                                             stream))


def kvq_prompt_workspace_size() -> int:
    return int(load().kvq_prompt_workspace_size())


def kvq_prompt_attention(args: kvq_prompt_args, ws: int, ws_bytes: int, stream: int = 0) -> None:
    _check("kvq_prompt_attention", load().kvq_prompt_attention(ctypes.byref(args), ws, ws_bytes, stream))
