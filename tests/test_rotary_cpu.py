"""The head norm with the rotation by position: refusals before anything is
launched, frequencies, fixed-point angles, and the reference's own checks; no GPU."""
from __future__ import annotations

import copy
import math
import pickle

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from io_aware_attention_fwd_gb300 import build_ext
from tests import rotary_ref as ref

FAKE = 0x10000  # aligned, non-null, never dereferenced on these paths
INVALID, UNSUPPORTED, ALIGNMENT = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_ALIGNMENT


@pytest.fixture(scope="module", autouse=True)
def built():
    build_ext.build()


def heads(ptr=FAKE, b=4096, s=512, h=64):
    return attn.attn_heads_t(ptr, b, s, h)


def rope(turns=FAKE, rot=64, inter=0, amp=1.0):
    return attn.attn_rotary_t(turns, rot, inter, amp)


REFUSALS = [
    (dict(B=-1), INVALID), (dict(S=-1), INVALID), (dict(H_q=0), INVALID), (dict(H_k=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(dtype=attn.ATTN_FP32), UNSUPPORTED), (dict(B=1 << 20, S=1 << 20), UNSUPPORTED), (dict(H_q=65536), UNSUPPORTED),
    (dict(S=1 << 32), INVALID), (dict(q=heads(None)), INVALID), (dict(k=None), INVALID), (dict(q=heads(FAKE + 8)), ALIGNMENT),
    (dict(k=heads(s=516)), ALIGNMENT), (dict(q=heads(h=68)), ALIGNMENT), (dict(k=heads(b=4)), ALIGNMENT),
    (dict(positions=None), INVALID), (dict(positions=FAKE + 2), ALIGNMENT), (dict(rope=rope(None)), INVALID),
    (dict(rope=rope(rot=72)), INVALID), (dict(rope=rope(rot=-16)), INVALID), (dict(rope=rope(rot=24)), UNSUPPORTED),
    (dict(rope=rope(inter=2)), INVALID), (dict(rope=rope(amp=math.nan)), INVALID), (dict(rope=rope(FAKE + 4)), ALIGNMENT),
    (dict(eps=-1.0), INVALID), (dict(eps=math.inf), INVALID), (dict(weight_dtype=attn.ATTN_FP16), UNSUPPORTED),
    (dict(weight_dtype=7), UNSUPPORTED), (dict(q_weight=FAKE + 1), ALIGNMENT),
    (dict(weight_dtype=attn.ATTN_FP32, k_weight=FAKE + 2), ALIGNMENT),
    (dict(B=0), attn.ATTN_OK), (dict(S=0, q=heads(None), positions=None), attn.ATTN_OK),
]


@pytest.mark.parametrize("kw,expect", REFUSALS + [(dict(q_out=None), INVALID), (dict(k_out=heads(FAKE + 2)), ALIGNMENT)])
def test_forward_argument_checks(kw, expect):
    args = dict(q=heads(), k=heads(), q_out=heads(), k_out=heads(), B=2, S=8, H_q=8, H_k=4, D=64, dtype=attn.ATTN_BF16, rope=rope(),
                positions=FAKE, q_weight=FAKE, k_weight=FAKE, weight_dtype=attn.ATTN_BF16, eps=1e-6)
    args.update(kw)
    assert attn.call_status(attn.attn_qk_norm_rope, **args) == expect


@pytest.mark.parametrize("kw,expect", [r for r in REFUSALS if r[1] != attn.ATTN_OK] + [
    (dict(dq_out=None), INVALID), (dict(dk=heads(None)), INVALID), (dict(dq_weight=None), INVALID), (dict(k_weight=None), INVALID),
    (dict(dk_weight=FAKE + 2), ALIGNMENT), (dict(workspace=FAKE + 8), ALIGNMENT), (dict(workspace=None), INVALID),
    (dict(workspace_bytes=64), INVALID),
    (dict(B=0, q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, workspace=None), attn.ATTN_OK),
])
def test_backward_argument_checks(kw, expect):
    args = dict(dq_out=heads(), dk_out=heads(), q=heads(), k=heads(), dq=heads(), dk=heads(), B=2, S=8, H_q=8, H_k=4, D=64,
                dtype=attn.ATTN_BF16, rope=rope(), positions=FAKE, q_weight=FAKE, k_weight=FAKE, weight_dtype=attn.ATTN_BF16,
                eps=1e-6, dq_weight=FAKE, dk_weight=FAKE, workspace=FAKE, workspace_bytes=1 << 30)
    args.update(kw)
    assert attn.call_status(attn.attn_qk_norm_rope_bwd, **args) == expect


def test_workspace_size():
    size = attn.attn_qk_norm_rope_bwd_workspace_bytes
    for bad in ((-1, 8, 4, 4, 64), (1, -8, 4, 4, 64), (1, 8, 0, 4, 64), (1, 8, 4, 4, 80), (1, 8, 4, 65536, 64), (1, 1 << 31, 4, 4, 64)):
        assert size(*bad) == 0
    # two rows of D sums a block, of which there are no more than the SMs hold at once
    assert size(1, 1, 1, 1, 64) == 2 * 64 * 4
    for rows in (1, 40, 8192, 1 << 20):
        n = size(2, rows, 32, 8, 128)
        assert n % (2 * 128 * 4) == 0 and 0 < n <= 8 * 152 * 2 * 128 * 4


def test_python_calls_check_their_tensors():
    q, k = torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    r = attn.Rotary([1.0] * 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        attn.qk_norm_rope(q, k, r, torch.zeros(8, dtype=torch.int32))
    with pytest.raises(TypeError):
        attn.qk_norm_rope(q.float(), k.float(), r, torch.zeros(8, dtype=torch.int32))
    for bad in (k[:7], k[None], k[..., :32], k[:, :0]):
        with pytest.raises(ValueError):
            attn.qk_norm_rope(q, bad, r, torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        attn.qk_norm_rope_backward(q, k, q, k, r, torch.zeros(8, dtype=torch.int32))
    for bad in ([1.0] * 7, [math.nan] * 8, [math.inf] * 8):
        with pytest.raises(ValueError):
            attn.Rotary(bad, device="cpu")
    with pytest.raises(ValueError):
        attn.Rotary([1.0] * 8, amplitude=math.nan, device="cpu")
    with pytest.raises(AttributeError):
        r.turns = None
    with pytest.raises(AttributeError):
        del r.turns


def test_rotary_copies():
    r = attn.Rotary([0.1 * i for i in range(16)], interleaved=True, amplitude=1.5, device="cpu")
    for c in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert torch.equal(c.turns, r.turns) and (c.rot, c.interleaved, c.amplitude) == (32, True, 1.5)
        assert c._c.turns == c.turns.data_ptr()


def test_angles_are_exact_modulo_a_turn():
    """position * turns modulo 2^64 is the angle, for positions of any size; Python's integers and a 50-digit pi tell."""
    from fractions import Fraction
    freqs = [1.0, 0.1, 3.5, -0.7, 1e-5, 1e-9, 0.0, 2 * math.pi]
    r = attn.Rotary(freqs, device="cpu")
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582")
    for f, t in zip(freqs, r.turns.tolist()):
        for pos in (0, 1, 77, 131071, 1 << 30, -5):
            got = (pos * t) % 2 ** 64
            want = (pos * Fraction(f) / two_pi) % 1
            off = abs(Fraction(got, 2 ** 64) - want)
            assert min(off, 1 - off) <= Fraction(max(1, abs(pos)), 2 ** 64)


def test_frequencies():
    f = attn.rotary_frequencies(64)
    assert len(f) == 32 and f[0] == 1.0 and math.isclose(f[-1], 10000 ** (-62 / 64))
    assert attn.rotary_frequencies(64, scaling="linear", factor=4.0) == [x / 4 for x in f]
    wide = attn.rotary_frequencies(64, scaling="base", factor=4.0)
    assert wide[0] == 1.0 and math.isclose(wide[-1], f[-1] / 4)
    parts = attn.rotary_frequencies(64, scaling="parts", factor=4.0, original_len=4096)
    for x, y in zip(f, parts):
        turns = 4096 * x / (2 * math.pi)
        if turns >= 32:
            assert y == x
        elif turns <= 1:
            assert math.isclose(y, x / 4)
        else:
            assert x / 4 < y < x
    for bad in (dict(rot=7), dict(rot=0), dict(rot=64, base=0.0), dict(rot=64, scaling="other"), dict(rot=64, factor=-1.0),
                dict(rot=64, scaling="parts", factor=2.0)):
        with pytest.raises(ValueError):
            attn.rotary_frequencies(**bad)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 64])
def test_reference_gradient_against_autograd_and_differences(rot, inter):
    g = torch.Generator().manual_seed(rot)
    x = torch.randn((3, 2, 64), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(64, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn((3, 2, 64), generator=g, dtype=torch.float64)
    pos, freqs = torch.tensor([0, 3, 1000]), attn.rotary_frequencies(rot) if rot else []

    def fwd(x, w):
        z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        return ref.turn(z, pos, freqs, inter, 1.3)

    fwd(x, w).backward(dy)
    ref.HALF_STEP.setdefault(torch.float64, 2.0 ** -53)
    ref.TINY.setdefault(torch.float64, 0.0)
    dx, _, dw, _ = ref.backward(dy, x.detach(), w.detach(), pos, freqs, inter, 1.3, 1e-6, 1)
    assert torch.allclose(dx, x.grad, rtol=1e-10, atol=1e-12) and torch.allclose(dw, w.grad, rtol=1e-10, atol=1e-12)
    # central differences along a direction
    ex, ew = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(64, generator=g, dtype=torch.float64)
    h = 1e-5
    with torch.no_grad():
        diff = ((fwd(x + h * ex, w + h * ew) - fwd(x - h * ex, w - h * ew)) / (2 * h) * dy).sum()
    assert math.isclose(float(diff), float((dx * ex).sum() + (dw * ew).sum()), rel_tol=1e-6)


def test_reference_turn_keeps_lengths_and_relative_angles():
    g = torch.Generator().manual_seed(5)
    x, y = torch.randn((2, 1, 1, 64), generator=g, dtype=torch.float64)
    f = attn.rotary_frequencies(32)
    for inter in (False, True):
        at = [ref.turn(z, torch.tensor([p]), f, inter, 1.0) for z, p in ((x, 7), (y, 3), (x, 1007), (y, 1003))]
        assert math.isclose(float((at[0] * at[1]).sum()), float((at[2] * at[3]).sum()), rel_tol=1e-9)
        assert math.isclose(float((at[0] ** 2).sum()), float((x ** 2).sum()), rel_tol=1e-12)
