"""Attention of up to 16 rows a key head over pages is as exact as from fp32 products: few
keys with small logits, where a P in one 16-bit term would show (test_token_ref_cpu.py)."""
from __future__ import annotations

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import token_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
LENS = [3, 8, 17, 40, 64, 5, 130, 700]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,new", [(8, 1), (16, 1), (5, 1), (8, 2), (1, 3), (4, 4)])
@pytest.mark.parametrize("shares", [False, True])  # a CTA a row, or the list of tiles and the merge
def test_as_exact_as_fp32(shares, G, new, d, dtype):
    H, page, pages = 2, 256, 8
    B = len(LENS)
    cache = attn.PagedKVCache.empty(B, H, B * pages, page, pages, d, dtype)
    cache.page_table.copy_(torch.arange(B * pages, dtype=torch.int32, device=DEV).view(B, pages))
    cache.length.copy_(torch.tensor(LENS, dtype=torch.int32))
    q = torch.empty((B * new, H * G, d), dtype=dtype, device=DEV)
    rows = []
    for b, n in enumerate(LENS):
        for h in range(H):
            x, k, v = ref.make(n, new * G, d, dtype, 100 * b + h, DEV)
            for j in range(0, n, page):
                e = min(n, j + page)
                cache.k_pages[b * pages + j // page, h, :e - j], cache.v_pages[b * pages + j // page, h, :e - j] = k[j:e], v[j:e]
            x = x.view(new, G, d)
            q[b * new:(b + 1) * new, h * G:(h + 1) * G] = x
            rows.append((b, h, n, x, k, v))
    starts = (torch.arange(B + 1, device=DEV) * new).int()
    o, lse = cache.attend(q, starts, max_new=new, max_len=2048 if shares else 1000)
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    for b, h, n, x, k, v in rows:
        for i in range(new):
            seen = n - new + i + 1
            heads = slice(h * G, (h + 1) * G)
            got, got_lse = o[b * new + i, heads], lse[b * new + i, heads]
            if seen <= 0:
                assert not got.any() and (got_lse == -torch.inf).all()
                continue
            want, want_lse, tol, lse_tol = ref.attend(x[i].double(), k[:seen].double(), v[:seen].double(), dtype, d ** -0.5)
            off = (got.double() - want).abs()
            assert (off <= tol).all(), (b, h, i, (off / tol).max())
            assert ((got_lse.double() - want_lse).abs() <= lse_tol).all()
