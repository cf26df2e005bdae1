"""The norm of query and key heads and the rotation by position, over the C ABI.

PyTorch provides the device memory and the stream; the computation is the CUDA
library's.
"""
from __future__ import annotations

import ctypes
import math

from . import _lib
from .api import current_handle, element_type, on_stream

# 2^256 / (2 pi), from 75 digits of pi
_TURN = 2 ** 256 * 10 ** 75 // (2 * 3141592653589793238462643383279502884197169399375105820974944592307816406286)


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_len: int | None = None, fast: float = 32.0, slow: float = 1.0) -> list[float]:
    """Radians a position of the rot // 2 pairs: base ** (-2 i / rot), slowed down for contexts
    that are `factor` times as long as a model was trained for.

    scaling: None; "linear", every frequency over the factor; "base", a base so much larger that
    the slowest pair is slowed by the factor and the fastest not at all; "parts" (B. Peng et al.,
    "YaRN: Efficient context window extension of large language models", 2023), pairs that make
    fewer than `slow` turns in original_len over the factor, those that make more than `fast` as
    they are, a linear ramp between.  That paper's amplitude, for Rotary, is 0.1 ln(factor) + 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even, 2 or more")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling == "parts":
        if original_len is None or not fast > slow:
            raise ValueError('scaling "parts" needs original_len, and fast above slow')
        keep = [min(1.0, max(0.0, (original_len * x / (2.0 * math.pi) - slow) / (fast - slow))) for x in f]
        return [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)]
    return f


class Rotary:
    """A rotation of heads by their token's position: the first 2 * len(frequencies) channels.

    frequencies: radians a position of each pair (floats; a multiple of 8 of them, or none).
    Pair i is channels (i, i + rot // 2), or (2 i, 2 i + 1) if interleaved.  amplitude: a
    factor on the turned channels.  The frequencies are held on the device as 64-bit fractions
    of a turn, so that angles are exact at every position.
    """

    __slots__ = ("frequencies", "turns", "rot", "interleaved", "amplitude", "device", "_c", "_address")

    def __init__(self, frequencies, interleaved: bool = False, amplitude: float = 1.0, device="cuda"):
        import torch

        f = tuple(float(x) for x in frequencies)
        if not all(math.isfinite(x) for x in f) or not math.isfinite(amplitude):
            raise ValueError("frequencies and amplitude must be finite")
        if len(f) % 8:
            raise ValueError("there must be a multiple of 8 frequencies (16 channels)")
        # f / (2 pi) * 2^64, rounded down, modulo 2^64: f is n / d exactly
        bits = [(n * _TURN // d >> 192) % 2 ** 64 for n, d in (x.as_integer_ratio() for x in f)]
        turns = torch.tensor([t - 2 ** 64 if t >> 63 else t for t in bits], dtype=torch.int64).to(device)
        fixed = object.__setattr__
        for name, value in (("frequencies", f), ("turns", turns), ("rot", 2 * len(f)), ("interleaved", bool(interleaved)),
                            ("amplitude", float(amplitude)), ("device", turns.device)):
            fixed(self, name, value)
        fixed(self, "_c", _lib.attn_rotary_t(turns.data_ptr() if f else None, self.rot, int(self.interleaved), self.amplitude))
        fixed(self, "_address", ctypes.addressof(self._c))

    def __setattr__(self, name, value):
        raise AttributeError("a Rotary does not change")

    def __delattr__(self, name):
        raise AttributeError("a Rotary does not change")

    def __reduce__(self):
        return type(self), (self.frequencies, self.interleaved, self.amplitude, self.device)


# As the serving calls, these are made once a layer and token: attributes are read once,
# addresses are passed as numbers, and the four rows' strides go over in one array.

def rope_address(rope, device):
    """The address of the struct a call passes on for a Rotary, or None."""
    if rope is None:
        return None
    if rope.device != device:
        raise ValueError(f"the rotation is on {rope.device}, the tensors are on {device}")
    return rope._address


def check_weight(w, dtype, index, D, name) -> int:
    """attn_dtype_t of a norm's weight."""
    import torch

    kind = w.dtype
    if w.shape != (D,) or w.get_device() != index or not w.is_contiguous() or (kind != dtype and kind != torch.float32):
        raise ValueError(f"{name} must be a contiguous tensor of {D} entries on device {index}, {dtype} or float32")
    return element_type(kind, True)


def norm_weights(q_weight, k_weight, dtype, index, D):
    """(address of q's, of k's, attn_dtype_t of both); index: the device's."""
    if q_weight is None:
        return None, *((None, _lib.ATTN_FP32) if k_weight is None else
                       (k_weight.data_ptr(), check_weight(k_weight, dtype, index, D, "k_weight")))
    code = check_weight(q_weight, dtype, index, D, "q_weight")
    if k_weight is None:
        return q_weight.data_ptr(), None, code
    if check_weight(k_weight, dtype, index, D, "k_weight") != code:
        raise TypeError("q_weight and k_weight must be of one type")
    return q_weight.data_ptr(), k_weight.data_ptr(), code


def _apart(b, B, s, S, h, H, D) -> bool:
    """Whether no two of B x S x H rows of D elements, at these strides, share an element."""
    heads, rows = h * (H - 1) + D, s * (S - 1) + D  # extents
    if (H < 2 or h >= D) and (S < 2 or s >= heads) and (B < 2 or b >= s * (S - 1) + heads):
        return True  # [B, S, H, D] and its slices
    if (S < 2 or s >= D) and (H < 2 or h >= rows) and (B < 2 or b >= h * (H - 1) + rows):
        return True  # [B, H, S, D]
    # any other layout: of every difference in the two shorter counts, the nearest in the longest
    (n1, s1), (n2, s2), (n3, s3) = sorted(((B, b), (S, s), (H, h)))
    for i in range(n1):
        for j in range(-(n2 - 1), n2):
            x = i * s1 + j * s2
            k = 0 if n3 < 2 or s3 == 0 else min(max(-x // s3, 1 - n3), n3 - 1)
            for c in (k, min(k + 1, n3 - 1)):
                if (i or j or c) and abs(x + c * s3) < D:
                    return False
    return True


def _strides(stride, shape, name, out=False):
    """(batch, row, head) strides of rows [S, H, D] or [B, S, H, D].  Where there is one of
    something, its stride says nothing (and may be anything).  out: its rows must lie apart."""
    if len(stride) == 4:
        b, s, h, one = stride
        B, S, H, D = shape
        if B < 2:
            b = 0
    else:
        s, h, one = stride
        S, H, D = shape
        B, b = 1, 0
    if S < 2:
        s = 0
    if H < 2:
        h = 0
    if one != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    if out and S and B and not _apart(b, B, s, S, h, H, D):
        raise ValueError(f"{name}: rows of an output must lie apart")
    return b, s, h


def _heads(t, shape, dtype, index, name, out=False):
    """What attn_heads_t holds of rows [S, H, D] or [B, S, H, D]: address, strides."""
    if t.dtype != dtype or t.get_device() != index or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor {tuple(shape)} on device {index}")
    return t.data_ptr(), *_strides(t.stride(), shape, name, out)


_Rows4 = ctypes.c_int64 * 16  # four attn_heads_t
_Rows6 = ctypes.c_int64 * 24


def _shapes(a, b):
    """(B, S, H_q, H_k, D) of rows [S, H, D] or [B, S, H, D]."""
    if len(a) not in (3, 4) or len(b) != len(a) or a[:-2] != b[:-2] or a[-1] != b[-1] or a[-2] < 1 or b[-2] < 1:
        raise ValueError("q and k must be [S, H, D] or [B, S, H, D] with the same rows and D")
    return (a[0] if len(a) == 4 else 1), a[-3], a[-2], b[-2], a[-1]


def _positions(positions, rope, shape, index):
    import torch

    if positions is None:
        if rope is not None and rope.rot:
            raise ValueError("positions are needed for a rotation")
        return None
    if positions.dtype != torch.int32 or positions.get_device() != index or positions.shape != shape or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous int32 tensor {tuple(shape)} on device {index}")
    return positions.data_ptr()


def qk_norm_rope(q, k, rope, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
                 stream=None):
    """q and k with every head normed, x / sqrt(mean(x^2) + eps) * weight, and turned by its position.

    q [S, H_q, D] or [B, S, H_q, D], k the same with H_k heads: bf16 or fp16 CUDA tensors, D 64 or
    128, the channels of a head contiguous and the other strides as they may be (multiples of 8
    elements): slices of a projection's output, or [B, H, S, D] tensors transposed.  rope: a
    Rotary, or None for no rotation.  positions: int32 [S] or [B, S].  q_weight, k_weight: [D] of
    q's type or float32; None: no norm of that one.  q_out, k_out: what to write to, of any
    strides that keep rows apart, q and k themselves among them (None: new contiguous tensors).
    Returns (q_out, k_out).
    """
    import torch

    shape, k_shape, dtype, device = q.shape, k.shape, q.dtype, q.device
    B, S, H_q, H_k, D = _shapes(shape, k_shape)
    code = element_type(dtype)
    if device.type != "cuda":
        raise ValueError("q and k must be CUDA tensors of one device")
    index = q.get_device()
    hq, hk = _strides(q.stride(), shape, "q"), _heads(k, k_shape, dtype, index, "k")
    r = rope_address(rope, device)
    pos = _positions(positions, rope, shape[:-2], index)
    qw, kw, w_code = norm_weights(q_weight, k_weight, dtype, index, D)
    handle = current_handle(device) if stream is None else None
    if handle is None:
        return on_stream(device, stream, lambda: qk_norm_rope(q, k, rope, positions, q_weight, k_weight, eps, q_out, k_out))
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=device)
    if k_out is None:
        k_out = torch.empty(k_shape, dtype=dtype, device=device)
    rows = _Rows4(q.data_ptr(), *hq, *hk, *_heads(q_out, shape, dtype, index, "q_out", True),
                  *_heads(k_out, k_shape, dtype, index, "k_out", True))
    at = ctypes.addressof(rows)
    _lib.attn_qk_norm_rope(at, at + 32, at + 64, at + 96, B, S, H_q, H_k, D, code, r, pos, qw, kw, w_code, eps, handle)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, rope, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                          dq=None, dk=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of qk_norm_rope for those of its results.

    dq_out, dk_out: of the shapes and type of q and k, strides as q and k may have them
    (attention_backward's [B, H, S, D] transposed, for instance).  The other arguments are the
    forward call's.  dq, dk: what to write to, as q_out and k_out there; dq_out and dk_out
    themselves will do.  The weights' gradients are float32 [D], None where there is no weight.
    """
    import torch

    shape, k_shape, dtype, device = q.shape, k.shape, q.dtype, q.device
    B, S, H_q, H_k, D = _shapes(shape, k_shape)
    code = element_type(dtype)
    if device.type != "cuda":
        raise ValueError("q and k must be CUDA tensors of one device")
    index = q.get_device()
    hq, hk = _strides(q.stride(), shape, "q"), _heads(k, k_shape, dtype, index, "k")
    gq, gk = _heads(dq_out, shape, dtype, index, "dq_out"), _heads(dk_out, k_shape, dtype, index, "dk_out")
    r = rope_address(rope, device)
    pos = _positions(positions, rope, shape[:-2], index)
    qw, kw, w_code = norm_weights(q_weight, k_weight, dtype, index, D)
    handle = current_handle(device) if stream is None else None
    if handle is None:
        return on_stream(device, stream, lambda: qk_norm_rope_backward(dq_out, dk_out, q, k, rope, positions, q_weight, k_weight,
                                                                       eps, dq, dk))
    if dq is None:
        dq = torch.empty(shape, dtype=dtype, device=device)
    if dk is None:
        dk = torch.empty(k_shape, dtype=dtype, device=device)
    dqw = None if qw is None else torch.empty(D, dtype=torch.float32, device=device)
    dkw = None if kw is None else torch.empty(D, dtype=torch.float32, device=device)
    ws, nbytes = None, 0
    if qw is not None or kw is not None:
        nbytes = _lib.attn_qk_norm_rope_bwd_workspace_bytes(B, S, H_q, H_k, D)
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    rows = _Rows6(*gq, *gk, q.data_ptr(), *hq, *hk, *_heads(dq, shape, dtype, index, "dq", True),
                  *_heads(dk, k_shape, dtype, index, "dk", True))
    at = ctypes.addressof(rows)
    _lib.attn_qk_norm_rope_bwd(at, at + 32, at + 64, at + 96, at + 128, at + 160, B, S, H_q, H_k, D, code, r, pos, qw, kw, w_code,
                               eps, dqw, dkw, ws, nbytes, handle)
    return dq, dk, dqw, dkw
