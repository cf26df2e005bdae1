"""Refusals of the paged cache's calls, before anything is launched, and their
reference's own checks; no GPU."""
from __future__ import annotations

import math

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


def pages(**kw):
    args = dict(k_pages=FAKE, v_pages=FAKE, page_table=FAKE, length=FAKE, B=3, H_kv=2, D=64, page=64, n_pages=20, max_pages=5,
                dtype=attn.ATTN_BF16)
    args.update(kw)
    return attn.attn_pages_t(**args)


APPEND = dict(k=FAKE, v=FAKE, rows=50, k_stride=128, v_stride=128, seq_start=FAKE, q=FAKE, q_stride=256, q_out=FAKE, H_q=4, rope=None,
              q_weight=FAKE, k_weight=FAKE, weight_dtype=attn.ATTN_BF16, eps=1e-6, length_out=FAKE)
ATTEND = dict(q=FAKE, q_stride=256, o=FAKE, lse=FAKE, rows=50, seq_start=FAKE, H_q=4, scale=0.125, window=0, sinks=0, max_new=50,
              max_len=320, workspace=FAKE, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,expect", [
    (dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID), (dict(page_table=None), INVALID), (dict(length=None), INVALID),
    (dict(B=0), INVALID), (dict(H_kv=0), INVALID), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(dtype=attn.ATTN_FP32), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(n_pages=1 << 30), UNSUPPORTED), (dict(max_pages=1 << 26), UNSUPPORTED), (dict(B=1 << 30), UNSUPPORTED),
    (dict(k_pages=FAKE + 8), ALIGNMENT), (dict(v_pages=FAKE + 2), ALIGNMENT), (dict(page_table=FAKE + 2), ALIGNMENT),
    (dict(length=FAKE + 1), ALIGNMENT),
])
def test_every_call_checks_the_cache(kw, expect):
    assert attn.call_status(attn.attn_paged_append, pages(**kw), **APPEND) == expect
    assert attn.call_status(attn.attn_paged_attend, pages(**kw), **ATTEND) == expect


def test_sizes_beyond_an_int():
    for name in ("B", "H_kv", "D", "page", "n_pages", "max_pages", "dtype"):
        with pytest.raises(OverflowError):
            pages(**{name: 1 << 32})
    for name in ("H_q", "window", "sinks", "max_new", "max_len"):
        assert attn.call_status(attn.attn_paged_attend, pages(), **{**ATTEND, name: (1 << 32) + 4}) == INVALID
    assert attn.call_status(attn.attn_paged_append, pages(), **{**APPEND, "H_q": (1 << 32) + 4}) == INVALID


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(rows=-1), INVALID), (dict(seq_start=None), INVALID),
    (dict(k_stride=120), INVALID), (dict(v_stride=0), INVALID), (dict(q_stride=248), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(H_q=0), INVALID), (dict(H_q=65536), UNSUPPORTED), (dict(length_out=None), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(k=FAKE + 8), ALIGNMENT), (dict(q_out=FAKE + 8), ALIGNMENT), (dict(k_stride=132), ALIGNMENT),
    (dict(q_stride=260), ALIGNMENT), (dict(seq_start=FAKE + 2), ALIGNMENT), (dict(length_out=FAKE + 2), ALIGNMENT),
    (dict(eps=math.nan), INVALID), (dict(weight_dtype=attn.ATTN_FP16), UNSUPPORTED), (dict(k_weight=FAKE + 1), ALIGNMENT),
    (dict(rope=attn.attn_rotary_t(FAKE, 24, 0, 1.0)), UNSUPPORTED), (dict(rope=attn.attn_rotary_t(None, 32, 0, 1.0)), INVALID),
    (dict(q=None, q_out=None), INVALID),  # a weight for queries that are not there
    (dict(length_out=FAKE + 4), INVALID), (dict(length_out=FAKE - 4), INVALID),  # over the old ones of other sequences
])
def test_append_argument_checks(kw, expect):
    assert attn.call_status(attn.attn_paged_append, pages(), **{**APPEND, **kw}) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(rows=-1), INVALID), (dict(seq_start=None), INVALID),
    (dict(H_q=0), INVALID), (dict(H_q=3, q_stride=256), INVALID), (dict(q_stride=248), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(max_new=-1), INVALID),
    (dict(max_len=-1), INVALID), (dict(max_len=321), INVALID), (dict(H_q=2 * 129, q_stride=2 * 129 * 64), UNSUPPORTED),
    (dict(rows=1 << 30), UNSUPPORTED), (dict(q=FAKE + 8), ALIGNMENT), (dict(q_stride=260), ALIGNMENT), (dict(o=FAKE + 8), ALIGNMENT),
    (dict(lse=FAKE + 2), ALIGNMENT), (dict(seq_start=FAKE + 1), ALIGNMENT), (dict(workspace=FAKE + 8), ALIGNMENT),
    (dict(rows=0), attn.ATTN_OK), (dict(rows=0, q=None, o=None, lse=None, workspace=None), attn.ATTN_OK), (dict(max_new=0), attn.ATTN_OK),
])
def test_attend_argument_checks(kw, expect):
    assert attn.call_status(attn.attn_paged_attend, pages(), **{**ATTEND, **kw}) == expect


def test_attend_needs_its_workspace():
    size = attn.attn_paged_attend_workspace_bytes
    c = pages(max_pages=200)
    for new in (1, 8, 50):
        n = size(3, 4, 2, 64, 50, new, 10000, 0, 0)
        assert n > 16
        for ws, nbytes in ((None, n), (FAKE, n - 1)):
            args = dict(ATTEND, max_new=new, max_len=10000, workspace=ws, workspace_bytes=nbytes)
            assert attn.call_status(attn.attn_paged_attend, c, **args) == INVALID
    assert size(3, 4, 2, 64, 3, 1, 700, 0, 0) == 16  # few short rows need none
    for bad in ((0, 4, 2, 64, 3, 1, 10, 0, 0), (1, 3, 2, 64, 3, 1, 10, 0, 0), (1, 4, 2, 80, 3, 1, 10, 0, 0), (1, 4, 2, 64, -1, 1, 10, 0, 0),
                (1, 4, 2, 64, 3, -1, 10, 0, 0), (1, 4, 2, 64, 3, 1, -1, 0, 0), (1, 258, 2, 64, 3, 1, 10, 0, 0),
                (1, 4, 2, 64, 3, 1, 10, -1, 0), (1, 4, 2, 64, 3, 1, 10, 0, -1)):
        assert size(*bad) == 0


def test_python_class_checks_its_buffers():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attn.PagedKVCache(k, k, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        attn.PagedKVCache.empty(1, 2, 4, 16, 2, 64, device="cpu")


def test_reference_attention_is_softmax():
    """Two sequences in pages against torch's float64 attention, with a window and sinks as a mask of its own."""
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn((2, 7, 2, 16, 64), generator=g).bfloat16()
    table = torch.tensor([[6, 2, 9, -1], [0, 3, 5, 1]], dtype=torch.int32)
    length = [30, 50]
    q = torch.randn((9, 4, 64), generator=g).bfloat16()
    for window, sinks in ((None, 0), (7, 0), (7, 3), (1, 1)):
        o, lse, _, _ = ref.attend(q, k, v, table, length, [0, 4, 9], 0.125, window, sinks)
        for b, (a, e) in enumerate(((0, 4), (4, 9))):
            n = length[b]
            kk, vv = (torch.cat([x[p].transpose(0, 1) for p in table[b, :-(-n // 16)].tolist()])[:n].double() for x in (k, v))
            mask = torch.zeros((e - a, n), dtype=torch.bool)
            for i in range(e - a):
                p = n - (e - a) + i
                for j in range(p + 1):
                    mask[i, j] = window is None or p - j < window or j < sinks
            full = torch.nn.functional.scaled_dot_product_attention(
                q[a:e].double().transpose(0, 1), kk.repeat_interleave(2, 1).transpose(0, 1), vv.repeat_interleave(2, 1).transpose(0, 1),
                attn_mask=mask, scale=0.125)
            assert torch.allclose(o[a:e].transpose(0, 1), full, atol=1e-12)
    # more new tokens than entries: the first ones see nothing
    o, lse, _, _ = ref.attend(q, k, v, table, [2, 50], [0, 4, 9], 0.125)
    assert not o[:2].any() and (lse[:2] == -math.inf).all() and torch.allclose(o[2], v[6, :, 0].double().repeat_interleave(2, 0))
