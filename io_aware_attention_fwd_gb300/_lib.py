"""ctypes binding of the C ABI declared in ``include/attn_fwd.h``.

Argument marshalling only: every step of the computation runs in the CUDA
library.  If the library has not been built, calls raise ``RuntimeError``;
there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import threading

from .build_ext import LIB_PATH

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_ALIGNMENT = 3
ATTN_ERR_LAUNCH = 4
ATTN_ERR_TIMEOUT = 5
ATTN_ERR_DEVICE = 6
ATTN_ERR_CAPACITY = 7

# attn_dtype_t
ATTN_BF16 = 0
ATTN_FP16 = 1
ATTN_FP32 = 2

# every extern "C" function include/attn_fwd.h declares
EXPORTED = ("attn_fwd", "attn_fwd_fp8", "attn_bwd", "attn_bwd_workspace_bytes", "attn_fwd_splitkv", "attn_fwd_splitkv_workspace_bytes",
            "attn_fwd_splitkv_suggest", "attn_fwd_schedule", "attn_merge", "attn_fwd_splitkv_static", "attn_status_str", "attn_fwd_debug_status",
            "attn_watchdog_selftest", "attn_fwd_abi_version", "attn_fwd_varlen", "attn_fwd_varlen_workspace_bytes",
            "attn_cache4_append", "attn_cache4_read", "attn_cache4_decode", "attn_cache4_decode_workspace_bytes",
            "attn_cache4_evict", "attn_cache4_evict_workspace_bytes")

_lock = threading.Lock()
_lib = None


_INT_MAX = 0x7FFFFFFF


def _int32(*values) -> bool:
    """Whether the values fit a C int.  ctypes would pass on their low 32 bits: a
    budget of 2^32 + 10, meant as no limit, would be one of 10."""
    return max(values) <= _INT_MAX and min(values) >= -_INT_MAX - 1


class attn_cache4_t(ctypes.Structure):
    """The struct of the same name: a 4-bit K/V cache's buffers and sizes."""

    _fields_ = [("k_codes", ctypes.c_void_p), ("k_meta", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_meta", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("length", ctypes.c_void_p), ("B", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("capacity", ctypes.c_int), ("D", ctypes.c_int)]

    def __setattr__(self, name, value):
        if name in ("B", "H_kv", "capacity", "D") and not _int32(value):
            raise OverflowError(f"attn_cache4_t.{name}: {value} does not fit an int")
        super().__setattr__(name, value)


class AttnError(RuntimeError):
    """A non-zero attn_status_t returned by the library."""

    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {attn_status_str(status)} (status {status})")


def load() -> ctypes.CDLL:
    """Load the built library (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not LIB_PATH.exists():
                raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                                   "(run __graft_entry__.build() or "
                                   "python -m io_aware_attention_fwd_gb300.build_ext)")
            lib = ctypes.CDLL(str(LIB_PATH))
            p, i = ctypes.c_void_p, ctypes.c_int
            lib.attn_fwd.restype = i
            lib.attn_fwd.argtypes = [p, p, p, p, p, i, i, i, i, i, ctypes.c_float, i, p, p]
            u64, i64 = ctypes.c_uint64, ctypes.c_int64
            lib.attn_fwd_splitkv.restype = i
            lib.attn_fwd_splitkv.argtypes = [p, p, p, p, p, i, i, i, i, i, ctypes.c_float, i, p, i, p, u64, p]
            lib.attn_fwd_splitkv_workspace_bytes.restype = u64
            lib.attn_fwd_splitkv_workspace_bytes.argtypes = [i, i, i, i, i]
            lib.attn_fwd_splitkv_suggest.restype = i
            lib.attn_fwd_splitkv_suggest.argtypes = [i, i, i, i, i, i]
            lib.attn_fwd_schedule.restype = i
            lib.attn_fwd_schedule.argtypes = [i, i, i, i, i, i, i, p, p, i]
            f = ctypes.c_float
            lib.attn_bwd.restype = i
            lib.attn_bwd.argtypes = [p, p, p, p, p, p, p, p, p, i, i, i, i, i, f, i, p, p, u64, p]
            lib.attn_bwd_workspace_bytes.restype = u64
            lib.attn_bwd_workspace_bytes.argtypes = [i, i, i, i]
            lib.attn_fwd_fp8.restype = i
            lib.attn_fwd_fp8.argtypes = [p, p, p, p, p, i, i, i, i, i, f, f, f, f, i, p, p]
            lib.attn_fwd_splitkv_static.restype = i
            lib.attn_fwd_splitkv_static.argtypes = [p, p, p, p, p, i, i, i, i, i, ctypes.c_float, i, p, i, p]
            lib.attn_merge.restype = i
            lib.attn_merge.argtypes = [p, p, i, i64, i, p, p, p]
            c4 = ctypes.POINTER(attn_cache4_t)
            lib.attn_fwd_varlen.restype = i
            lib.attn_fwd_varlen.argtypes = [p, p, p, p, p, i64, p, i, i, i, i, i, i64, i64, i64, f, i, p, u64, p]
            lib.attn_fwd_varlen_workspace_bytes.restype = u64
            lib.attn_fwd_varlen_workspace_bytes.argtypes = [i64, i, i, i, i]
            lib.attn_cache4_append.restype = i
            lib.attn_cache4_append.argtypes = [c4, p, p, i64, i64, i64, i, p, p, p, p]
            lib.attn_cache4_read.restype = i
            lib.attn_cache4_read.argtypes = [c4, p, p, i64, i64, i64, i, p, p, p]
            lib.attn_cache4_decode.restype = i
            lib.attn_cache4_decode.argtypes = [c4, p, i64, p, p, i, i, f, i, p, p, p, u64, p]
            lib.attn_cache4_decode_workspace_bytes.restype = u64
            lib.attn_cache4_decode_workspace_bytes.argtypes = [i, i, i, i, i, i]
            lib.attn_cache4_evict.restype = i
            lib.attn_cache4_evict.argtypes = [c4, i, i, i, p, p, p, p, u64, p]
            lib.attn_cache4_evict_workspace_bytes.restype = u64
            lib.attn_cache4_evict_workspace_bytes.argtypes = [i, i, i, i]
            lib.attn_status_str.restype = ctypes.c_char_p
            lib.attn_status_str.argtypes = [i]
            lib.attn_fwd_debug_status.restype = i
            lib.attn_fwd_debug_status.argtypes = [p]
            lib.attn_watchdog_selftest.restype = i
            lib.attn_watchdog_selftest.argtypes = [ctypes.c_uint64, p]
            lib.attn_fwd_abi_version.restype = i
            lib.attn_fwd_abi_version.argtypes = []
            _lib = lib
    return _lib


def _addr(x):
    """Device address of a tensor-like (``data_ptr()``) or a plain int/None."""
    if x is None or type(x) is int:
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _stream(s):
    if s is None or type(s) is int:
        return s
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


def attn_status_str(status: int) -> str:
    return load().attn_status_str(int(status)).decode()


def attn_fwd(q, k, v, o, lse, B: int, H: int, S_q: int, S_kv: int, D: int, scale: float,
             causal: bool, kv_valid_len=None, stream=None) -> None:
    """Enqueue the attention forward pass (see include/attn_fwd.h).

    q, k, v, o, lse, kv_valid_len: device buffers (tensors or raw addresses).
    Raises AttnError on a non-zero status.
    """
    st = load().attn_fwd(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), int(B), int(H),
                         int(S_q), int(S_kv), int(D), float(scale), int(bool(causal)),
                         _addr(kv_valid_len), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd")


def attn_fwd_fp8(q, k, v, o, lse, B: int, H: int, S_q: int, S_kv: int, D: int, scale: float,
                 q_descale: float, k_descale: float, v_descale: float, causal: bool,
                 kv_valid_len=None, stream=None) -> None:
    """Enqueue the FP8 (e4m3) forward pass (see include/attn_fwd.h)."""
    st = load().attn_fwd_fp8(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), int(B), int(H),
                             int(S_q), int(S_kv), int(D), float(scale), float(q_descale),
                             float(k_descale), float(v_descale), int(bool(causal)),
                             _addr(kv_valid_len), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_fp8")


def attn_bwd(q, k, v, o, lse, d_o, dq, dk, dv, B: int, H: int, S_q: int, S_kv: int, D: int,
             scale: float, causal: bool, kv_valid_len, workspace, workspace_bytes: int,
             stream=None) -> None:
    """Enqueue the backward pass (see include/attn_fwd.h)."""
    st = load().attn_bwd(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(d_o), _addr(dq),
                         _addr(dk), _addr(dv), int(B), int(H), int(S_q), int(S_kv), int(D),
                         float(scale), int(bool(causal)), _addr(kv_valid_len), _addr(workspace),
                         int(workspace_bytes), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd")


def attn_bwd_workspace_bytes(B: int, H: int, S_q: int, D: int) -> int:
    return int(load().attn_bwd_workspace_bytes(int(B), int(H), int(S_q), int(D)))


def attn_fwd_splitkv(q, k, v, o, lse, B: int, H: int, S_q: int, S_kv: int, D: int, scale: float,
                     causal: bool, kv_valid_len, n_splits: int, workspace, workspace_bytes: int,
                     stream=None) -> None:
    """Enqueue the key-split forward pass (see include/attn_fwd.h)."""
    st = load().attn_fwd_splitkv(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), int(B), int(H),
                                 int(S_q), int(S_kv), int(D), float(scale), int(bool(causal)),
                                 _addr(kv_valid_len), int(n_splits), _addr(workspace),
                                 int(workspace_bytes), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_splitkv")


def attn_fwd_splitkv_workspace_bytes(B: int, H: int, S_q: int, D: int, n_splits: int) -> int:
    return int(load().attn_fwd_splitkv_workspace_bytes(int(B), int(H), int(S_q), int(D), int(n_splits)))


def attn_fwd_splitkv_suggest(B: int, H: int, S_q: int, S_kv: int, D: int, causal: bool) -> int:
    return int(load().attn_fwd_splitkv_suggest(int(B), int(H), int(S_q), int(S_kv), int(D),
                                               int(bool(causal))))


def attn_fwd_schedule(B: int, H: int, S_q: int, S_kv: int, D: int, elem_bytes: int, sms: int):
    """The host-built unit order of a causal launch of this shape (see
    include/attn_fwd.h): (off, unit) as lists, CTA c running
    unit[off[c]:off[c + 1]]; None where the launch has no such order."""
    n_pairs = -(-int(S_q) // 256)
    cap = max(1, int(B) * int(H) * n_pairs)
    off = (ctypes.c_uint16 * (max(1, int(sms)) + 1))()
    unit = (ctypes.c_uint16 * cap)()
    n = load().attn_fwd_schedule(int(B), int(H), int(S_q), int(S_kv), int(D), int(elem_bytes), int(sms),
                                 ctypes.addressof(off), ctypes.addressof(unit), cap)
    if n < 0:
        raise ValueError("attn_fwd_schedule: invalid arguments")
    if n == 0:
        return None
    G = min(n, int(sms))
    return list(off[:G + 1]), list(unit[:n])


def attn_merge(o_parts, lse_parts, n_parts: int, rows: int, D: int, o, lse, stream=None) -> None:
    """Enqueue the log-sum-exp merge of per-key-set results (see include/attn_fwd.h)."""
    st = load().attn_merge(_addr(o_parts), _addr(lse_parts), int(n_parts), int(rows), int(D),
                           _addr(o), _addr(lse), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_merge")


# Size of the library's fixed scratch (ATTN_STATIC_SCRATCH_BYTES in the header).
STATIC_SCRATCH_BYTES = 32 << 20


def attn_fwd_splitkv_static(q, k, v, o, lse, B: int, H: int, S_q: int, S_kv: int, D: int,
                            scale: float, causal: bool, kv_valid_len, n_splits: int,
                            stream=None) -> None:
    """Key-split forward using the library's fixed scratch instead of a
    workspace, for callers that cannot allocate device memory (see
    include/attn_fwd.h: 32 MiB cap, one call at a time on the GPU)."""
    st = load().attn_fwd_splitkv_static(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), int(B),
                                        int(H), int(S_q), int(S_kv), int(D), float(scale),
                                        int(bool(causal)), _addr(kv_valid_len), int(n_splits),
                                        _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_splitkv_static")


def attn_fwd_varlen(q, k, v, o, lse, total: int, seq_start, n_seqs: int, H_q: int, H_kv: int, D: int, dtype: int,
                    q_stride: int, k_stride: int, v_stride: int, scale: float, causal: bool, workspace,
                    workspace_bytes: int, stream=None) -> None:
    """Enqueue attention over packed prompts with grouped heads (see include/attn_fwd.h)."""
    if not _int32(n_seqs, H_q, H_kv, D, dtype):
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_fwd_varlen")
    st = load().attn_fwd_varlen(_addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), total, _addr(seq_start), n_seqs, H_q,
                                H_kv, D, dtype, q_stride, k_stride, v_stride, scale, int(bool(causal)),
                                _addr(workspace), workspace_bytes, _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_varlen")


@functools.lru_cache(maxsize=256)
def attn_fwd_varlen_workspace_bytes(total: int, n_seqs: int, H_q: int, H_kv: int, D: int) -> int:
    return load().attn_fwd_varlen_workspace_bytes(total, n_seqs, H_q, H_kv, D) if _int32(n_seqs, H_q, H_kv, D) else 0


def attn_cache4_append(cache: attn_cache4_t, k, v, rows: int, k_stride: int, v_stride: int, dtype: int, seq_start,
                       first_pos, length_out, stream=None) -> None:
    """Enqueue the quantising append of K and V rows (see include/attn_fwd.h)."""
    st = load().attn_cache4_append(cache, _addr(k), _addr(v), rows, k_stride, v_stride, dtype, _addr(seq_start),
                                   _addr(first_pos), _addr(length_out), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_cache4_append")


def attn_cache4_read(cache: attn_cache4_t, k, v, rows: int, k_stride: int, v_stride: int, dtype: int, seq_start,
                     first_slot, stream=None) -> None:
    """Enqueue the read-back of cache entries (see include/attn_fwd.h)."""
    st = load().attn_cache4_read(cache, _addr(k), _addr(v), rows, k_stride, v_stride, dtype, _addr(seq_start),
                                 _addr(first_slot), _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_cache4_read")


def attn_cache4_decode(cache: attn_cache4_t, q, q_stride: int, o, lse, H_q: int, dtype: int, scale: float,
                       max_len: int, weight_in, weight_out, workspace, workspace_bytes: int, stream=None) -> None:
    """Enqueue attention of one token per sequence over the cache (see include/attn_fwd.h)."""
    if not _int32(H_q, dtype, max_len):
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_cache4_decode")
    st = load().attn_cache4_decode(cache, _addr(q), q_stride, _addr(o), _addr(lse), H_q, dtype, scale, max_len,
                                   _addr(weight_in), _addr(weight_out), _addr(workspace), workspace_bytes,
                                   _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_cache4_decode")


@functools.lru_cache(maxsize=256)
def attn_cache4_decode_workspace_bytes(B: int, H_q: int, H_kv: int, D: int, max_len: int, with_weight: bool) -> int:
    if not _int32(B, H_q, H_kv, D, max_len):
        return 0
    return load().attn_cache4_decode_workspace_bytes(B, H_q, H_kv, D, max_len, int(bool(with_weight)))


def attn_cache4_evict(cache: attn_cache4_t, budget: int, recent: int, max_len: int, weight_out, pos_out, length_out,
                      workspace, workspace_bytes: int, stream=None) -> None:
    """Enqueue the eviction by accumulated weight (see include/attn_fwd.h)."""
    if not _int32(budget, recent, max_len):
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_cache4_evict")
    st = load().attn_cache4_evict(cache, budget, recent, max_len, _addr(weight_out), _addr(pos_out), _addr(length_out),
                                  _addr(workspace), workspace_bytes, _stream(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_cache4_evict")


@functools.lru_cache(maxsize=256)
def attn_cache4_evict_workspace_bytes(B: int, H_kv: int, max_len: int, budget: int) -> int:
    return load().attn_cache4_evict_workspace_bytes(B, H_kv, max_len, budget) if _int32(B, H_kv, max_len, budget) else 0


def call_status(fn, *args, **kwargs) -> int:
    """Run one of the raising wrappers above and return its status instead."""
    try:
        fn(*args, **kwargs)
    except AttnError as e:
        return e.status
    return ATTN_OK


def attn_fwd_status(*args, **kwargs) -> int:
    """Same as attn_fwd but returns the raw status instead of raising."""
    try:
        attn_fwd(*args, **kwargs)
    except AttnError as e:
        return e.status
    return ATTN_OK


def attn_fwd_debug_status(stream=None) -> int:
    return int(load().attn_fwd_debug_status(_stream(stream)))


def attn_watchdog_selftest(timeout_ns: int, stream=None) -> int:
    return int(load().attn_watchdog_selftest(int(timeout_ns), _stream(stream)))


def attn_fwd_abi_version() -> int:
    return int(load().attn_fwd_abi_version())
