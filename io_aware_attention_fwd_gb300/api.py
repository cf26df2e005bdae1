"""Tensor-level convenience wrapper over the C ABI.

PyTorch only provides the device memory and the stream here; the computation
is the CUDA library's.
"""
from __future__ import annotations

import math

from . import _lib


def attention_forward(q, k, v, scale: float | None = None, causal: bool = False,
                      kv_valid_len=None, out=None, lse=None, stream=None, n_splits: int | None = None):
    """O and LSE for bf16 CUDA tensors q [B,H,S_q,D], k/v [B,H,S_kv,D].

    kv_valid_len: int32 CUDA tensor [B] or None.  n_splits: key chunks (None
    picks attn_fwd_splitkv_suggest's count; more than 1 takes a torch-allocated
    workspace).  Returns (o, lse) with o bf16 [B,H,S_q,D] and lse fp32 [B,H,S_q].
    """
    import torch

    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("q, k, v must be bfloat16")
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("q, k, v must be CUDA tensors")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous [B,H,S,D]")
    B, H, S_q, D = q.shape
    S_kv = k.shape[2]
    if tuple(k.shape) != (B, H, S_kv, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B,H,S_kv,D] matching q")
    if kv_valid_len is not None:
        if kv_valid_len.dtype != torch.int32 or not kv_valid_len.is_cuda or kv_valid_len.numel() != B:
            raise ValueError("kv_valid_len must be an int32 CUDA tensor with B entries")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, S_q), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    if n_splits is None:
        n_splits = _lib.attn_fwd_splitkv_suggest(B, H, S_q, S_kv, D, causal)
    if n_splits > 1:
        nbytes = _lib.attn_fwd_splitkv_workspace_bytes(B, H, S_q, D, n_splits)
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
        _lib.attn_fwd_splitkv(q, k, v, out, lse, B, H, S_q, S_kv, D, scale, causal, kv_valid_len,
                              n_splits, ws, nbytes, stream)
    else:
        _lib.attn_fwd(q, k, v, out, lse, B, H, S_q, S_kv, D, scale, causal, kv_valid_len, stream)
    return out, lse


def attention_backward(q, k, v, o, lse, d_o, scale: float | None = None, causal: bool = False,
                       kv_valid_len=None, stream=None):
    """dQ, dK, dV (bf16) for the forward pass that produced (o, lse) from q, k, v.

    All tensors are contiguous CUDA tensors as attention_forward uses them; d_o
    is bf16 [B,H,S_q,D].  The fp32 workspace comes from torch's allocator.
    """
    import torch

    B, H, S_q, D = q.shape
    S_kv = k.shape[2]
    for t in (q, k, v, o, d_o):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v, o, d_o must be contiguous bf16 CUDA tensors")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = _lib.attn_bwd_workspace_bytes(B, H, S_q, D)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    _lib.attn_bwd(q, k, v, o, lse, d_o, dq, dk, dv, B, H, S_q, S_kv, D, scale, causal, kv_valid_len,
                  ws, nbytes, stream)
    return dq, dk, dv


# The serving calls are made once a layer and token, and for few tokens their
# time on the host is what counts (the GPU's is 3 to 8 us): attributes are read
# once, addresses are passed as numbers, and the stream is taken as the handle
# that torch keeps (a Stream object costs 3 us to make).

def current_handle(device):
    """The current stream's handle where `device` is the current one, else None."""
    import torch

    index = device.index
    return torch._C._cuda_getCurrentRawStream(index) if torch._C._cuda_getDevice() == index else None


def on_stream(device, stream, call):
    """call() with `device` current and, where a stream is given, that stream
    too, so that what the call allocates belongs to it."""
    import torch

    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.device(device):
        if stream is None:
            return call()
        if not isinstance(stream, torch.cuda.Stream):
            handle = _lib._stream(stream)
            stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
        with torch.cuda.stream(stream):
            return call()


_TYPES = {}  # torch dtype -> attn_dtype_t


def element_type(dtype, also_fp32: bool = False) -> int:
    """attn_dtype_t of a torch dtype the serving calls take."""
    if not _TYPES:
        import torch

        _TYPES.update({torch.bfloat16: _lib.ATTN_BF16, torch.float16: _lib.ATTN_FP16, torch.float32: _lib.ATTN_FP32})
    code = _TYPES.get(dtype, -1)
    if code < 0 or (code == _lib.ATTN_FP32 and not also_fp32):
        raise TypeError(f"{dtype}: must be bfloat16 or float16" + (" or float32" if also_fp32 else ""))
    return code


def row_stride(t, shape, name: str) -> int:
    """Elements from one row of t [rows, H, D] to the next; the heads of a row lie side by side."""
    s = t.stride()
    rows, H, D = shape
    if (s[2] != 1 and D > 1) or (s[1] != D and H > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return s[0] if rows > 1 else H * D


def check_out(t, shape, dtype, device, name: str) -> None:
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {device}")


def check_int32(t, n: int, device, name: str) -> None:
    import torch

    if t.shape != (n,) or t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on {device}")


def attention_varlen(q, k, v, seq_start, scale: float | None = None, causal: bool = True, out=None, lse=None,
                     stream=None):
    """O and LSE of whole prompts packed one behind the other, with grouped heads.

    q [total, H_q, D], k and v [total, H_kv, D]: bf16 or fp16 CUDA tensors (all
    of one type) whose rows may lie apart, as slices of one projection's output
    do; H_q is a multiple of H_kv, D is 64 or 128.  seq_start: int32 CUDA tensor
    [n + 1], sequence s being rows seq_start[s] .. seq_start[s + 1] - 1; query
    head h sees key head h // (H_q // H_kv) of its own sequence, up to its own
    row if causal.  Returns (o, lse): o [total, H_q, D] of q's type, lse fp32
    [H_q, total].  Rows that belong to no sequence are left as they were, which
    in outputs allocated here means undefined.
    """
    import torch

    shape, k_shape = q.shape, k.shape
    if len(shape) != 3 or len(k_shape) != 3 or v.shape != k_shape:
        raise ValueError("q must be [total, H_q, D], k and v [total, H_kv, D]")
    total, H_q, D = shape
    H_kv = k_shape[1]
    if k_shape[0] != total or k_shape[2] != D or H_kv < 1 or H_q % H_kv:
        raise ValueError("k and v must be [total, H_kv, D] matching q, H_q a multiple of H_kv")
    dtype, device = q.dtype, q.device
    code = element_type(dtype)
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k, v must be of one type")
    if device.type != "cuda" or k.device != device or v.device != device:
        raise ValueError("q, k, v must be CUDA tensors of one device")
    n = seq_start.numel() - 1
    if n < 1:
        raise ValueError("seq_start must have at least two entries")
    check_int32(seq_start, n + 1, device, "seq_start")
    q_stride, k_stride, v_stride = row_stride(q, shape, "q"), row_stride(k, k_shape, "k"), row_stride(v, k_shape, "v")
    if out is not None:
        check_out(out, shape, dtype, device, "out")
    if lse is not None:
        check_out(lse, (H_q, total), torch.float32, device, "lse")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    handle = current_handle(device) if stream is None else None
    if handle is None:
        return on_stream(device, stream, lambda: attention_varlen(q, k, v, seq_start, scale, causal, out, lse))
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    if lse is None:
        lse = torch.empty((H_q, total), dtype=torch.float32, device=device)
    nbytes = _lib.attn_fwd_varlen_workspace_bytes(total, n, H_q, H_kv, D)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 16 else None
    _lib.attn_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), total,
                         seq_start.data_ptr(), n, H_q, H_kv, D, code, q_stride, k_stride, v_stride, scale, causal, ws,
                         nbytes, handle)
    return out, lse
