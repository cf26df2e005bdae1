"""A K/V cache held in 4 bits, over the C ABI.

PyTorch provides the device memory and the stream; the computation is the CUDA
library's.
"""
from __future__ import annotations

import math

from . import _lib
from .api import check_int32, check_out, current_handle, element_type, on_stream, row_stride

GROUP = 64  # channels that share a scale and a minimum


class KVCache4:
    """K and V of ``B`` sequences and ``H_kv`` key heads, ``capacity`` entries each.

    Every 64 channels of a K or V row share a bf16 scale and minimum, and a value
    is a code in 0 .. 15 that stands for code * scale + minimum (4.5 bits a value;
    include/attn_fwd.h has the format).  The buffers are plain tensors:

      k_codes, v_codes  uint8 [B, H_kv, capacity, D // 2]
      k_meta, v_meta    bf16  [B, H_kv, capacity, D // 64, 2]
      weight            fp32  [B, H_kv, capacity]  attention weight received
      pos               int32 [B, H_kv, capacity]  position of the entry's token
      length            int32 [B]                  entries held

    The calls work in place on these buffers, on the current stream (or the one
    given), and never wait for the GPU.  Where a call has ``..._out`` arguments,
    what it would update in place goes there instead; assigned to the cache
    (``cache.length = length_out``), those buffers are then the cache after the
    call.  A buffer may be exchanged for another of the same shape, type and device;
    the sizes are fixed.  ``copy.copy`` gives a cache over the same buffers,
    ``copy.deepcopy`` one over copies of them.
    """

    __slots__ = ("k_codes", "k_meta", "v_codes", "v_meta", "weight", "pos", "length", "B", "H_kv", "capacity", "D",
                 "device", "_c", "_layout")

    def __init__(self, k_codes, k_meta, v_codes, v_meta, weight, pos, length):
        import torch

        if k_codes.dim() != 4 or not k_codes.is_cuda:
            raise ValueError("k_codes must be a CUDA tensor [B, H_kv, capacity, D // 2]")
        B, H_kv, capacity, half = k_codes.shape
        D, device = 2 * half, k_codes.device
        if D % GROUP:
            raise ValueError(f"D must be a multiple of {GROUP}")
        codes, meta, entry = (B, H_kv, capacity, half), (B, H_kv, capacity, D // GROUP, 2), (B, H_kv, capacity)
        fixed = object.__setattr__
        fixed(self, "B", B)
        fixed(self, "H_kv", H_kv)
        fixed(self, "capacity", capacity)
        fixed(self, "D", D)
        fixed(self, "device", device)
        fixed(self, "_c", _lib.attn_cache4_t(B=B, H_kv=H_kv, capacity=capacity, D=D))
        fixed(self, "_layout", {"k_codes": (codes, torch.uint8), "v_codes": (codes, torch.uint8),
                                "k_meta": (meta, torch.bfloat16), "v_meta": (meta, torch.bfloat16),
                                "weight": (entry, torch.float32), "pos": (entry, torch.int32), "length": ((B,), torch.int32)})
        self.k_codes, self.k_meta, self.v_codes, self.v_meta = k_codes, k_meta, v_codes, v_meta
        self.weight, self.pos, self.length = weight, pos, length

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
        return type(self), (self.k_codes, self.k_meta, self.v_codes, self.v_meta, self.weight, self.pos, self.length)

    @classmethod
    def empty(cls, B: int, H_kv: int, capacity: int, D: int, device="cuda") -> "KVCache4":
        """An empty cache; its memory is allocated here."""
        import torch

        if D not in (64, 128):
            raise ValueError("D must be 64 or 128")
        # an allocation each: a half of one for K and V begins off an 8-byte boundary
        # where D is 64 and the number of entries odd
        codes = [torch.empty((B, H_kv, capacity, D // 2), dtype=torch.uint8, device=device) for _ in range(2)]
        meta = [torch.empty((B, H_kv, capacity, D // GROUP, 2), dtype=torch.bfloat16, device=device) for _ in range(2)]
        return cls(codes[0], meta[0], codes[1], meta[1],
                   torch.zeros((B, H_kv, capacity), dtype=torch.float32, device=device),
                   torch.zeros((B, H_kv, capacity), dtype=torch.int32, device=device),
                   torch.zeros(B, dtype=torch.int32, device=device))

    def _rows(self, k, v, seq_start, also_fp32=False):
        shape, device, dtype = k.shape, self.device, k.dtype
        if len(shape) != 3 or v.shape != shape or shape[1] != self.H_kv or shape[2] != self.D:
            raise ValueError(f"k and v must be [rows, {self.H_kv}, {self.D}]")
        if k.device != device or v.device != device:
            raise ValueError(f"k and v must be on {device}")
        if v.dtype != dtype:
            raise TypeError("k and v must be of one type")
        rows = shape[0]
        if seq_start is not None:
            check_int32(seq_start, self.B + 1, device, "seq_start")
        elif rows != self.B:
            raise ValueError(f"without seq_start k and v have one row for each of the {self.B} sequences")
        return rows, row_stride(k, shape, "k"), row_stride(v, shape, "v"), element_type(dtype, also_fp32)

    def append(self, k, v, seq_start=None, first_pos=None, length_out=None, stream=None) -> None:
        """Quantise rows of K and V (bf16 or fp16, [rows, H_kv, D]) into the next entries.

        seq_start: int32 [B + 1], rows seq_start[b] .. seq_start[b + 1] - 1 being
        sequence b's; None: one row for each sequence.  first_pos: int32 [B],
        position of each sequence's first new token (None: its slot's number).
        The new entries' weights are 0.  Rows beyond the capacity are dropped, and
        attn_fwd_debug_status then reports ATTN_ERR_CAPACITY (once, for whichever
        cache of the device it was).
        """
        rows, ks, vs, code = self._rows(k, v, seq_start)
        device = self.device
        if first_pos is not None:
            check_int32(first_pos, self.B, device, "first_pos")
        if length_out is None:
            length_out = self.length
        else:
            check_int32(length_out, self.B, device, "length_out")
        handle = current_handle(device) if stream is None else None
        if handle is None:
            return on_stream(device, stream, lambda: self.append(k, v, seq_start, first_pos, length_out))
        _lib.attn_cache4_append(self._c, k.data_ptr(), v.data_ptr(), rows, ks, vs, code, seq_start, first_pos,
                                length_out.data_ptr(), handle)

    def read(self, seq_start=None, rows: int | None = None, first_slot=None, dtype=None, k_out=None, v_out=None,
             stream=None):
        """The values entries stand for, as packed rows (k, v) [rows, H_kv, D].

        Row i of sequence b is its slot first_slot[b] + i (None: slot i); seq_start
        as append takes it.  k_out and v_out (bf16, fp16 or fp32), or `rows` and
        `dtype` (bfloat16 if None) for new tensors.  Rows of slots outside the
        capacity and rows of no sequence are left as they were (zero in new
        tensors).
        """
        if (k_out is None) != (v_out is None):
            raise ValueError("k_out and v_out go together")
        if k_out is None and rows is None:
            if seq_start is not None:
                raise ValueError("rows is needed with seq_start where k_out and v_out are not given")
            rows = self.B
        device = self.device
        if first_slot is not None:
            check_int32(first_slot, self.B, device, "first_slot")
        handle = current_handle(device) if stream is None else None
        if handle is None:
            return on_stream(device, stream, lambda: self.read(seq_start, rows, first_slot, dtype, k_out, v_out))
        if k_out is None:
            import torch

            k_out, v_out = torch.zeros((2, rows, self.H_kv, self.D), dtype=dtype or torch.bfloat16, device=device)
        n, ks, vs, code = self._rows(k_out, v_out, seq_start, True)
        _lib.attn_cache4_read(self._c, k_out.data_ptr(), v_out.data_ptr(), n, ks, vs, code, seq_start, first_slot, handle)
        return k_out, v_out

    def attend(self, q, scale: float | None = None, weight_out=None, max_len: int | None = None, out=None, lse=None,
               stream=None):
        """Attention of one token per sequence, q [B, H_q, D] (bf16 or fp16), over its entries.

        weight_out: where not None, the entries' weights plus what this token gave
        each, summed over the query heads of its key head; pass ``cache.weight`` to
        add in place.  max_len: a bound on the lengths, which are clamped to it
        (None: the capacity); it sizes the workspace and picks the kernel, so a
        close one pays where the capacity is much larger than what is held.  Returns (o, lse): o
        [B, H_q, D] of q's type, lse fp32 [B, H_q]; 0 and -inf for a sequence
        without entries.
        """
        import torch

        B, D, device, dtype, shape = self.B, self.D, self.device, q.dtype, q.shape
        if len(shape) != 3 or shape[0] != B or shape[2] != D or shape[1] < 1 or shape[1] % self.H_kv:
            raise ValueError(f"q must be [{B}, H_q, {D}], H_q a multiple of {self.H_kv}")
        if q.device != device:
            raise ValueError(f"q must be on {device}")
        H_q, code, stride = shape[1], element_type(dtype), row_stride(q, shape, "q")
        if weight_out is not None:
            check_out(weight_out, self.weight.shape, torch.float32, device, "weight_out")
        if out is not None:
            check_out(out, shape, dtype, device, "out")
        if lse is not None:
            check_out(lse, (B, H_q), torch.float32, device, "lse")
        if max_len is None:
            max_len = self.capacity
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        handle = current_handle(device) if stream is None else None
        if handle is None:
            return on_stream(device, stream, lambda: self.attend(q, scale, weight_out, max_len, out, lse))
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=device)
        if lse is None:
            lse = torch.empty((B, H_q), dtype=torch.float32, device=device)
        nbytes = _lib.attn_cache4_decode_workspace_bytes(B, H_q, self.H_kv, D, max_len, weight_out is not None)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 16 else None
        _lib.attn_cache4_decode(self._c, q.data_ptr(), stride, out.data_ptr(), lse.data_ptr(), H_q, code, scale, max_len,
                                None if weight_out is None else self.weight, weight_out, ws, nbytes, handle)
        return out, lse

    def evict(self, budget: int, recent: int = 0, weight_out=None, pos_out=None, length_out=None,
              max_len: int | None = None, stream=None) -> None:
        """Shorten every sequence to at most `budget` entries.

        Each key head keeps the entries of the `recent` newest positions, then
        those of the highest weight (ties: the lower slot).  Kept entries from
        behind the budget move into the slots that became free; attention does not
        depend on the entries' order.  max_len: as attend takes it, at most 393216
        (or the budget); entries behind it are dropped, and it picks the kernel.
        """
        import torch

        B, device, entry = self.B, self.device, self.weight.shape
        if weight_out is None:
            weight_out = self.weight
        else:
            check_out(weight_out, entry, torch.float32, device, "weight_out")
        if pos_out is None:
            pos_out = self.pos
        else:
            check_out(pos_out, entry, torch.int32, device, "pos_out")
        if length_out is None:
            length_out = self.length
        else:
            check_int32(length_out, B, device, "length_out")
        if max_len is None:
            max_len = self.capacity
        handle = current_handle(device) if stream is None else None
        if handle is None:
            return on_stream(device, stream, lambda: self.evict(budget, recent, weight_out, pos_out, length_out, max_len))
        nbytes = _lib.attn_cache4_evict_workspace_bytes(B, self.H_kv, max_len, budget)
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
        _lib.attn_cache4_evict(self._c, budget, recent, max_len, weight_out.data_ptr(), pos_out.data_ptr(),
                               length_out.data_ptr(), ws.data_ptr(), nbytes, handle)
