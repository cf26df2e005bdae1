"""A step without tokens through the paged cache, with everything that may go with it."""
from __future__ import annotations

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("q_weight", [False, True])
@pytest.mark.parametrize("k_weight", [False, True])
@pytest.mark.parametrize("turned", [False, True])
def test_no_tokens(turned, k_weight, q_weight, out):
    cache = attn.PagedKVCache.empty(2, 2, 4, 16, 2, 64)
    cache.k_pages.fill_(3.0), cache.v_pages.fill_(4.0)
    cache.page_table.copy_(torch.tensor([[0, 1], [2, 3]], dtype=torch.int32))
    cache.length.copy_(torch.tensor([7, 3], dtype=torch.int32))
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    e, q = (torch.empty((0, h, 64), dtype=torch.bfloat16, device=DEV) for h in (2, 8))
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    length_out = torch.full((2,), -1, dtype=torch.int32, device=DEV) if out else None
    got = cache.append(e, e, seq_start=s, q=q, rope=attn.Rotary(attn.rotary_frequencies(64)) if turned else None,
                       q_weight=w if q_weight else None, k_weight=w if k_weight else None, q_out=torch.empty_like(q) if out else None,
                       length_out=length_out)
    o, lse = cache.attend(got, s)
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    assert got.shape == q.shape and o.shape == q.shape and lse.shape == (0, 8)
    assert (length_out if out else cache.length).tolist() == [7, 3]
    assert (cache.k_pages == 3.0).all() and (cache.v_pages == 4.0).all()
