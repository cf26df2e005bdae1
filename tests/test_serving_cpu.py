"""Refusals of the serving calls (packed prompts, 4-bit cache), before
anything is launched, and their references' own checks; no GPU."""
from __future__ import annotations

import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from io_aware_attention_fwd_gb300 import build_ext
from tests import serving_ref as ref

FAKE = 0x10000  # aligned, non-null, never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def built():
    build_ext.build()


INVALID, UNSUPPORTED, ALIGNMENT = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_ALIGNMENT


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(lse=None), INVALID), (dict(seq_start=None), INVALID), (dict(total=-1), INVALID),
    (dict(total=9000, workspace=None), INVALID), (dict(total=9000, workspace_bytes=16 + 12 * 73 - 1), INVALID), (dict(n_seqs=0), INVALID),
    (dict(H_kv=0), INVALID), (dict(H_q=6), INVALID), (dict(H_q=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(q_stride=8 * 64 - 8), INVALID), (dict(k_stride=4 * 64 - 8), INVALID), (dict(v_stride=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(dtype=attn.ATTN_FP32), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED),
    (dict(H_q=4 * 129, q_stride=4 * 129 * 64), UNSUPPORTED), (dict(total=1 << 31), UNSUPPORTED),
    (dict(q=FAKE + 2), ALIGNMENT), (dict(o=FAKE + 8), ALIGNMENT), (dict(lse=FAKE + 2), ALIGNMENT),
    (dict(seq_start=FAKE + 1), ALIGNMENT), (dict(workspace=FAKE + 8), ALIGNMENT),
    (dict(q_stride=8 * 64 + 4), ALIGNMENT), (dict(v_stride=4 * 64 + 1), ALIGNMENT),
    (dict(total=0), attn.ATTN_OK), (dict(total=0, q=None, seq_start=None, workspace=None), attn.ATTN_OK),
])
def test_varlen_argument_checks(kw, expect):
    args = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, total=100, seq_start=FAKE, n_seqs=3, H_q=8, H_kv=4, D=64,
                dtype=attn.ATTN_BF16, q_stride=8 * 64, k_stride=4 * 64, v_stride=4 * 64, scale=0.125, causal=True,
                workspace=FAKE, workspace_bytes=attn.attn_fwd_varlen_workspace_bytes(100, 3, 8, 4, 64))
    args.update(kw)
    assert attn.call_status(attn.attn_fwd_varlen, **args) == expect


def test_varlen_workspace_size():
    # a header, then 12 bytes for every 2 * (128 / G) tokens and one ragged unit a sequence
    assert attn.attn_fwd_varlen_workspace_bytes(1000, 7, 32, 8, 128) == 16 + 12 * (1000 // 64 + 7)
    # none where those units, of every key head, are no more than 152
    assert attn.attn_fwd_varlen_workspace_bytes(1000, 4, 32, 8, 128) == 16
    assert attn.attn_fwd_varlen_workspace_bytes(1000, 5, 32, 8, 128) == 16 + 12 * (1000 // 64 + 5)
    for bad in ((-1, 1, 8, 8, 64), (10, 0, 8, 8, 64), (10, 1, 8, 3, 64), (10, 1, 8, 8, 96), (10, 1, 129, 1, 64)):
        assert attn.attn_fwd_varlen_workspace_bytes(*bad) == 0


def cache(**kw):
    args = dict(k_codes=FAKE, k_meta=FAKE, v_codes=FAKE, v_meta=FAKE, weight=FAKE, pos=FAKE, length=FAKE, B=3, H_kv=2,
                capacity=100, D=64)
    args.update(kw)
    return attn.attn_cache4_t(*args.values())


CACHE_REFUSALS = [
    (dict(k_codes=None), INVALID), (dict(v_codes=None), INVALID), (dict(k_meta=None), INVALID),
    (dict(v_meta=None), INVALID), (dict(length=None), INVALID), (dict(B=0), INVALID), (dict(H_kv=0), INVALID),
    (dict(capacity=0), INVALID), (dict(D=32), UNSUPPORTED), (dict(B=1 << 20, H_kv=1 << 10), UNSUPPORTED),
    (dict(k_codes=FAKE + 8), ALIGNMENT), (dict(v_meta=FAKE + 2), ALIGNMENT), (dict(length=FAKE + 1), ALIGNMENT),
    (dict(weight=FAKE + 2), ALIGNMENT), (dict(pos=FAKE + 2), ALIGNMENT),
]


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS)
def test_every_cache_call_checks_the_cache(kw, expect):
    c = cache(**kw)
    assert attn.call_status(attn.attn_cache4_append, c, FAKE, FAKE, 3, 128, 128, 0, None, None, FAKE) == expect
    assert attn.call_status(attn.attn_cache4_read, c, FAKE, FAKE, 3, 128, 128, 0, None, None) == expect
    assert attn.call_status(attn.attn_cache4_decode, c, FAKE, 256, FAKE, FAKE, 4, 0, 0.1, 100, None, None, FAKE, 1 << 40) == expect
    assert attn.call_status(attn.attn_cache4_evict, c, 10, 2, 100, FAKE, FAKE, FAKE, FAKE, 1 << 40) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(rows=-1), INVALID),
    (dict(seq_start=None, rows=4), INVALID), (dict(k_stride=120), INVALID), (dict(v_stride=0), INVALID),
    (dict(length_out=None), INVALID), (dict(dtype=attn.ATTN_FP32), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(k=FAKE + 8), ALIGNMENT), (dict(k_stride=132), ALIGNMENT), (dict(seq_start=FAKE + 2), ALIGNMENT),
    (dict(first_pos=FAKE + 2), ALIGNMENT), (dict(length_out=FAKE + 2), ALIGNMENT),
])
def test_append_argument_checks(kw, expect):
    args = dict(k=FAKE, v=FAKE, rows=50, k_stride=128, v_stride=128, dtype=attn.ATTN_BF16, seq_start=FAKE,
                first_pos=None, length_out=FAKE)
    args.update(kw)
    assert attn.call_status(attn.attn_cache4_append, cache(), **args) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INVALID), (dict(rows=-1), INVALID), (dict(seq_start=None), INVALID), (dict(v_stride=64), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(v=FAKE + 4), ALIGNMENT), (dict(k_stride=130), ALIGNMENT),
    (dict(dtype=attn.ATTN_FP32, k_stride=130), ALIGNMENT), (dict(first_slot=FAKE + 2), ALIGNMENT),
    (dict(rows=0, k=None, v=None), attn.ATTN_OK),
])
def test_read_argument_checks(kw, expect):
    args = dict(k=FAKE, v=FAKE, rows=50, k_stride=128, v_stride=128, dtype=attn.ATTN_FP16, seq_start=FAKE, first_slot=None)
    args.update(kw)
    assert attn.call_status(attn.attn_cache4_read, cache(), **args) == expect


WEIGHTS = dict(weight_in=FAKE, weight_out=FAKE)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(workspace=None, **WEIGHTS), INVALID),
    (dict(H_q=3, q_stride=256), INVALID), (dict(H_q=0), INVALID),
    (dict(q_stride=248), INVALID), (dict(max_len=0), INVALID), (dict(max_len=101), INVALID),
    (dict(scale=-1.0), INVALID), (dict(weight_in=FAKE), INVALID), (dict(weight_out=FAKE), INVALID),
    (dict(**WEIGHTS), INVALID),  # the workspace lacks the scores' room
    (dict(dtype=attn.ATTN_FP32), UNSUPPORTED), (dict(H_q=2 * 129, q_stride=2 * 129 * 64), UNSUPPORTED),
    (dict(q=FAKE + 8), ALIGNMENT), (dict(q_stride=260), ALIGNMENT), (dict(o=FAKE + 8), ALIGNMENT),
    (dict(workspace=FAKE + 4), ALIGNMENT),
])
def test_decode_argument_checks(kw, expect):
    args = dict(q=FAKE, q_stride=256, o=FAKE, lse=FAKE, H_q=4, dtype=attn.ATTN_BF16, scale=0.1, max_len=100,
                weight_in=None, weight_out=None, workspace=FAKE,
                workspace_bytes=attn.attn_cache4_decode_workspace_bytes(3, 4, 2, 64, 100, False))
    args.update(kw)
    assert attn.call_status(attn.attn_cache4_decode, cache(), **args) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(budget=0), INVALID), (dict(recent=-1), INVALID), (dict(recent=11), INVALID), (dict(max_len=0), INVALID),
    (dict(max_len=101), INVALID), (dict(weight_out=None), INVALID), (dict(pos_out=None), INVALID),
    (dict(length_out=None), INVALID), (dict(workspace=None), INVALID), (dict(workspace_bytes=100), INVALID),
    (dict(weight_out=FAKE + 2), ALIGNMENT), (dict(workspace=FAKE + 8), ALIGNMENT),
])
def test_evict_argument_checks(kw, expect):
    args = dict(budget=10, recent=2, max_len=100, weight_out=FAKE, pos_out=FAKE, length_out=FAKE, workspace=FAKE,
                workspace_bytes=attn.attn_cache4_evict_workspace_bytes(3, 2, 100, 10))
    args.update(kw)
    assert attn.call_status(attn.attn_cache4_evict, cache(), **args) == expect


def test_evict_longest_sequences():
    n = 393216
    c = cache(capacity=n + 1)
    size = attn.attn_cache4_evict_workspace_bytes(3, 2, n, 10)
    assert size == 3 * 2 * 2 * 10 * 4 and attn.attn_cache4_evict_workspace_bytes(3, 2, n + 1, 10) == 0
    for budget, status in ((10, UNSUPPORTED), (n, UNSUPPORTED)):
        assert attn.call_status(attn.attn_cache4_evict, c, budget, 0, n + 1, FAKE, FAKE, FAKE, FAKE, 1 << 40) == status


def test_evict_needs_weights_and_positions():
    n = attn.attn_cache4_evict_workspace_bytes(3, 2, 100, 10)
    for kw in (dict(weight=None), dict(pos=None)):
        assert attn.call_status(attn.attn_cache4_evict, cache(**kw), 10, 2, 100, FAKE, FAKE, FAKE, FAKE, n) == INVALID


def test_workspace_sizes_refuse_what_the_calls_refuse():
    for bad in ((0, 4, 2, 64, 10, 0), (1, 3, 2, 64, 10, 0), (1, 4, 2, 80, 10, 0), (1, 4, 2, 64, 0, 0), (1, 258, 2, 64, 10, 0)):
        assert attn.attn_cache4_decode_workspace_bytes(*bad) == 0
    for bad in ((0, 1, 10, 5), (1, 0, 10, 5), (1, 1, 0, 5), (1, 1, 10, 0)):
        assert attn.attn_cache4_evict_workspace_bytes(*bad) == 0
    # scores of every 64-key tile and query head come on top
    a, b = (attn.attn_cache4_decode_workspace_bytes(2, 24, 8, 128, 5000, w) for w in (0, 1))
    assert b - a == 2 * 8 * 79 * 3 * 64 * 4
    # none for short caches without weights
    assert attn.attn_cache4_decode_workspace_bytes(2, 24, 8, 128, 2048, 0) == 16
    assert attn.attn_cache4_decode_workspace_bytes(2, 24, 8, 128, 2049, 0) > 16


def test_long_caches_need_the_decode_workspace():
    n = attn.attn_cache4_decode_workspace_bytes(3, 4, 2, 64, 2500, False)
    args = dict(q=FAKE, q_stride=256, o=FAKE, lse=FAKE, H_q=4, dtype=0, scale=0.1, max_len=2500, weight_in=None, weight_out=None)
    for ws, nbytes in ((None, n), (FAKE, n - 1)):
        assert attn.call_status(attn.attn_cache4_decode, cache(capacity=2500), workspace=ws, workspace_bytes=nbytes, **args) == INVALID


def test_python_calls_check_their_tensors():
    q, k = torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    start = torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attention_varlen(q, k, k, start)
    with pytest.raises(TypeError):
        attn.attention_varlen(q.float(), k.float(), k.float(), start)
    with pytest.raises(ValueError):
        attn.attention_varlen(q, k[:7], k[:7], start)
    with pytest.raises(ValueError):
        attn.attention_varlen(q[:, :3], k, k, start)
    c = torch.zeros(1, 2, 8, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        attn.KVCache4(c, c, c, c, c, c, c)
    with pytest.raises(ValueError):
        attn.KVCache4.empty(1, 1, 8, 96, device="cpu")


def test_reference_format_worked_example():
    """0 .. 15 over a group reproduces itself; a constant group has s = 0; a value half way goes to the even code."""
    x = torch.arange(64, dtype=torch.float64) % 16
    c, s, m = ref.quantise(x[None])
    assert torch.equal(c[0], x) and float(s[0]) == 1.0 and float(m[0]) == 0.0
    c, s, m = ref.quantise(torch.full((1, 64), 2.5))
    assert float(s[0]) == 0.0 and float(m[0]) == 2.5 and not c.any()
    x[:2] = torch.tensor([2.5, 3.5])
    assert ref.quantise(x[None])[0][0, :2].tolist() == [2.0, 4.0]
    codes = ref.pack(ref.quantise(x[None])[0])
    assert codes[0, 0] == 2 | 4 << 4
    assert torch.equal(ref.unpack(codes), ref.quantise(x[None])[0])


def test_reference_eviction_worked_example():
    # budget 3 of 6, the newest position protected: slot 4 (newest), then weights 9 (slot 5) and 5 (slot 1)
    w, p = [1.0, 5.0, 2.0, 3.0, 0.0, 9.0], [0, 1, 2, 3, 9, 5]
    assert ref.evict(w, p, 6, 3, 1) == [4, 1, 5]
    assert ref.evict(w, p, 6, 6, 1) == [0, 1, 2, 3, 4, 5]
    assert ref.evict([1.0] * 5, list(range(5)), 5, 2, 0) == [0, 1]
    assert ref.evict([1.0, math.nan, 2.0], [0, 1, 2], 3, 1, 0) == [1]


def test_reference_attention_is_softmax():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((5, h, 64), generator=g).bfloat16() for h in (4, 2, 2))
    o, lse, _, _ = ref.varlen(q, k, v, [0, 2, 2, 5], 0.125, True)
    full = torch.nn.functional.scaled_dot_product_attention(
        q[2:, :].double().transpose(0, 1), k[2:].double().repeat_interleave(2, 1).transpose(0, 1),
        v[2:].double().repeat_interleave(2, 1).transpose(0, 1), is_causal=True, scale=0.125)
    assert torch.allclose(o[2:].transpose(0, 1), full, atol=1e-12)
    assert torch.allclose(o[0], v[0].double().repeat_interleave(2, 0))
    assert torch.allclose(lse[:, 0], (q[0].double() * k[0].double().repeat_interleave(2, 0)).sum(-1) * 0.125)
