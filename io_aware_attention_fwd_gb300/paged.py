"""A K/V cache in pages, over the C ABI.

PyTorch provides the device memory and the stream; the computation is the CUDA
library's.
"""
from __future__ import annotations

import math

from . import _lib
from .api import check_int32, check_out, current_handle, element_type, on_stream, row_stride
from .rotary import norm_weights, rope_address


class PagedKVCache:
    """K and V of ``B`` sequences in pages that a table hands out.

    Entry j of sequence b, the token at position j, is row j % page of page
    page_table[b, j // page].  The buffers are plain tensors:

      k_pages, v_pages  bf16 or fp16 [n_pages, H_kv, page, D], page 16 .. 256 a power of two
      page_table        int32 [B, max_pages]  places that no entry needs may hold anything
      length            int32 [B]             entries held

    Which pages a sequence has is the caller's to say, by writing page_table; sequences may
    share pages that neither writes.  A place that is needed and names no page: append drops
    the entry, attend takes K and V as zeros, and attn_fwd_debug_status reports ATTN_ERR_PAGE
    (once, for whichever cache of the device it was).  The calls work in place on these
    buffers, on the current stream (or the one given), and never wait for the GPU.  A buffer
    may be exchanged for another of the same shape, type and device; ``copy.copy`` gives a
    cache over the same buffers, ``copy.deepcopy`` one over copies of them.
    """

    __slots__ = ("k_pages", "v_pages", "page_table", "length", "B", "H_kv", "D", "page", "n_pages", "max_pages", "dtype",
                 "device", "_c", "_layout")

    def __init__(self, k_pages, v_pages, page_table, length):
        import torch

        if k_pages.dim() != 4 or not k_pages.is_cuda:
            raise ValueError("k_pages must be a CUDA tensor [n_pages, H_kv, page, D]")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [B, max_pages]")
        n_pages, H_kv, page, D = k_pages.shape
        B, max_pages = page_table.shape
        device, dtype = k_pages.device, k_pages.dtype
        code = element_type(dtype)
        if page not in (16, 32, 64, 128, 256):
            raise ValueError("a page must have 16, 32, 64, 128 or 256 rows")
        fixed = object.__setattr__
        for name, value in (("B", B), ("H_kv", H_kv), ("D", D), ("page", page), ("n_pages", n_pages), ("max_pages", max_pages),
                            ("dtype", dtype), ("device", device)):
            fixed(self, name, value)
        fixed(self, "_c", _lib.attn_pages_t(B=B, H_kv=H_kv, D=D, page=page, n_pages=n_pages, max_pages=max_pages, dtype=code))
        rows = tuple(k_pages.shape)
        fixed(self, "_layout", {"k_pages": (rows, dtype), "v_pages": (rows, dtype),
                                "page_table": ((B, max_pages), torch.int32), "length": ((B,), torch.int32)})
        self.k_pages, self.v_pages, self.page_table, self.length = k_pages, v_pages, page_table, length

    def __setattr__(self, name, value):
        """A buffer, checked; the struct that the calls pass on holds its address."""
        import torch

        layout = self._layout.get(name)
        if layout is None:
            raise AttributeError(f"a cache's {name} cannot be set")
        if not isinstance(value, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        check_out(value, *layout, self.device, name)
        object.__setattr__(self, name, value)
        setattr(self._c, name, value.data_ptr())

    def __delattr__(self, name):
        raise AttributeError(f"a cache's {name} cannot be removed")

    def __reduce__(self):
        return type(self), (self.k_pages, self.v_pages, self.page_table, self.length)

    @classmethod
    def empty(cls, B: int, H_kv: int, n_pages: int, page: int, max_pages: int, D: int, dtype=None, device="cuda") -> "PagedKVCache":
        """Pages that no sequence has yet (the table is all -1, the lengths 0); their memory is allocated here."""
        import torch

        k, v = (torch.empty((n_pages, H_kv, page, D), dtype=dtype or torch.bfloat16, device=device) for _ in range(2))
        return cls(k, v, torch.full((B, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(B, dtype=torch.int32, device=device))

    def append(self, k, v, seq_start=None, q=None, rope=None, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None,
               length_out=None, stream=None):
        """Write rows of K and V ([rows, H_kv, D], the cache's type) into the next entries.

        seq_start: int32 [B + 1], rows seq_start[b] .. seq_start[b + 1] - 1 being sequence b's;
        None: one row for each sequence.  rope, q_weight, k_weight, eps: as qk_norm_rope takes
        them; K, and the tokens' queries q [rows, H_q, D] if given, are normed and turned by
        their entries' numbers on the way.  Returns q_out (a new tensor if None; rows of no
        sequence are left as they were), or None without q.  length_out: where the new lengths
        go (None: ``length`` itself, which it must not overlap in part).  Rows beyond the capacity (max_pages * page) are dropped,
        and attn_fwd_debug_status then reports ATTN_ERR_CAPACITY.
        """
        import torch

        shape, device, dtype, D = k.shape, self.device, self.dtype, self.D
        if len(shape) != 3 or v.shape != shape or shape[1] != self.H_kv or shape[2] != D:
            raise ValueError(f"k and v must be [rows, {self.H_kv}, {D}]")
        if k.device != device or v.device != device:
            raise ValueError(f"k and v must be on {device}")
        if k.dtype != dtype or v.dtype != dtype:
            raise TypeError(f"k and v must be {dtype}, as the cache is")
        rows = shape[0]
        if seq_start is not None:
            check_int32(seq_start, self.B + 1, device, "seq_start")
        elif rows != self.B:
            raise ValueError(f"without seq_start k and v have one row for each of the {self.B} sequences")
        H_q, q_stride = 0, 0
        if q is not None:
            q_shape = q.shape
            if len(q_shape) != 3 or q_shape[0] != rows or q_shape[2] != D or q_shape[1] < 1:
                raise ValueError(f"q must be [{rows}, H_q, {D}]")
            if q.dtype != dtype or q.device != device:
                raise ValueError(f"q must be {dtype} on {device}")
            H_q, q_stride = q_shape[1], row_stride(q, q_shape, "q")
            if q_out is not None:
                check_out(q_out, q_shape, dtype, device, "q_out")
        elif q_out is not None or q_weight is not None:
            raise ValueError("q_out and q_weight go with q")
        r = rope_address(rope, device)
        qw, kw, w_code = norm_weights(q_weight, k_weight, dtype, device.index, D)
        if length_out is None:
            length_out = self.length
        else:
            check_int32(length_out, self.B, device, "length_out")
        k_stride, v_stride = row_stride(k, shape, "k"), row_stride(v, shape, "v")
        handle = current_handle(device) if stream is None else None
        if handle is None:
            return on_stream(device, stream, lambda: self.append(k, v, seq_start, q, rope, q_weight, k_weight, eps, q_out, length_out))
        if q is not None and q_out is None:
            q_out = torch.empty(q_shape, dtype=dtype, device=device)
        _lib.attn_paged_append(self._c, k.data_ptr(), v.data_ptr(), rows, k_stride, v_stride, seq_start, q, q_stride, q_out, H_q, r,
                               qw, kw, w_code, eps, length_out.data_ptr(), handle)
        return q_out

    def attend(self, q, seq_start=None, scale: float | None = None, window: int | None = None, sinks: int = 0,
               max_new: int | None = None, max_len: int | None = None, out=None, lse=None, stream=None):
        """Attention of new tokens, q [rows, H_q, D] of the cache's type, over the entries held.

        A sequence's rows are its newest entries (append first, then attend): of n, the i-th has
        position length - n + i and sees entry j if j <= position and (there is no window, or
        j > position - window, or j < sinks).  seq_start: int32 [B + 1] as append takes it; None:
        one row for each sequence.  max_new and max_len: bounds on a sequence's rows and length
        (None: the rows there are, the capacity).  Rows behind max_new are left as they were,
        lengths are clamped to max_len; both pick the kernel and size the workspace, so close
        ones pay.  Pages that no token sees are not read.  Returns (o, lse): o of q's shape and
        type, lse fp32 [rows, H_q]; 0 and -inf for a token that sees nothing.  Rows of no
        sequence are left as they were, which in outputs allocated here means undefined.
        """
        import torch

        shape, device, dtype, D, B, H_kv = q.shape, self.device, self.dtype, self.D, self.B, self.H_kv
        if len(shape) != 3 or shape[2] != D or shape[1] < 1 or shape[1] % H_kv:
            raise ValueError(f"q must be [rows, H_q, {D}], H_q a multiple of {H_kv}")
        if q.device != device:
            raise ValueError(f"q must be on {device}")
        if q.dtype != dtype:
            raise TypeError(f"q must be {dtype}, as the cache is")
        rows, H_q = shape[0], shape[1]
        if seq_start is not None:
            check_int32(seq_start, B + 1, device, "seq_start")
        elif rows != B:
            raise ValueError(f"without seq_start q has one row for each of the {B} sequences")
        if window is None:
            window = 0
        elif window < 1:
            raise ValueError("window must be 1 or more, or None")
        if max_new is None:
            max_new = rows if seq_start is not None else 1
        if max_len is None:
            max_len = self.max_pages * self.page
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        stride = row_stride(q, shape, "q")
        if out is not None:
            check_out(out, shape, dtype, device, "out")
        if lse is not None:
            check_out(lse, (rows, H_q), torch.float32, device, "lse")
        handle = current_handle(device) if stream is None else None
        if handle is None:
            return on_stream(device, stream, lambda: self.attend(q, seq_start, scale, window or None, sinks, max_new, max_len, out, lse))
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=device)
        if lse is None:
            lse = torch.empty((rows, H_q), dtype=torch.float32, device=device)
        nbytes = _lib.attn_paged_attend_workspace_bytes(B, H_q, H_kv, D, rows, min(max_new, rows), max_len, window, sinks)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 16 else None
        _lib.attn_paged_attend(self._c, q.data_ptr(), stride, out.data_ptr(), lse.data_ptr(), rows, seq_start, H_q, scale, window,
                               sinks, max_new, max_len, ws, nbytes, handle)
        return out, lse
