"""fp16 chunks over pages through the list of units and the merge, units cut by one share
and by several; fp16 windows, of chunks and of single tokens, over long contexts."""
from __future__ import annotations

import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import rotary_ref as ref
from tests.test_paged_gpu import attend, make_cache, queries, starts_of

pytestmark = pytest.mark.gpu

DEV = "cuda"


def size(cache, rows, hq, new, max_len, window=0, sinks=0):
    return attn.attn_paged_attend_workspace_bytes(cache.B, hq, cache.H_kv, cache.D, rows, new, max_len, window, sinks)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,hq,H,page", [(64, 8, 2, 16), (128, 8, 2, 64), (128, 8, 1, 256), (64, 10, 2, 32)])
@pytest.mark.parametrize("new,had", [([60], [9000]), ([300], [5000]), ([200, 0, 33, 128], [4000, 900, 2500, 0]), ([700, 700], [100, 3000])], ids=str)
def test_through_the_list(new, had, d, hq, H, page, dtype):
    cache = make_cache([a + b for a, b in zip(had, new)], [0] * len(new), H, d, page, dtype, seed=d + page)
    starts, _ = starts_of(new)
    q = queries(starts[-1] + 3, hq, d, dtype)
    most = cache.max_pages * page
    assert size(cache, q.shape[0], hq, max(new), most) > 16
    attend(cache, q, starts)
    if max(had) >= 4000:
        for window, sinks in ((3000, 5), (2500, 700)):
            assert size(cache, q.shape[0], hq, max(new), most, window, sinks) > 16
            attend(cache, q, starts, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("new", [3, 60])
@pytest.mark.parametrize("d", [64, 128])
def test_one_unit_cut_by_many_shares(d, new, dtype):
    """One sequence, one key head, many keys: nearly every SM has a piece of the one unit."""
    cache = make_cache([20000 + new], [0], 1, d, 64, dtype, seed=new)
    attend(cache, queries(new, 8, d, dtype), [0, new], max_new=new)


def test_values_that_span_fp16():
    """V up to fp16's largest number and keys many nats apart, joined by the merge: finite, and with their bits."""
    d, new, n = 64, 40, 6000
    cache = make_cache([n], [0], 1, d, 64, torch.float16, seed=3)
    table = cache.page_table[0, :-(-n // 64)].long()
    for x, p in enumerate(table.tolist()):
        cache.k_pages[p] *= 0.05 + 0.02 * (x % 50)
        cache.v_pages[p] = 60000.0 if x % 3 == 0 else -60000.0 if x % 3 == 1 else cache.v_pages[p]
    for q in (queries(new, 4, d, torch.float16), torch.zeros((new, 4, d), dtype=torch.float16, device=DEV)):
        attend(cache, q, [0, new], scale=0.3)
    cache.v_pages.fill_(65504.0)
    o, _ = cache.attend(queries(new, 4, d, torch.float16), torch.tensor([0, new], dtype=torch.int32, device=DEV))
    assert (o.float() >= 65440.0).all() and o.isfinite().all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("window,sinks", [(700, 4), (4096, 64), (1, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_of_single_tokens(d, window, sinks, dtype):
    lens = [12000, 700, 699, 4097, 0, 9001]
    cache = make_cache(lens, [0] * len(lens), 2, d, 16, dtype, seed=window)
    attend(cache, queries(len(lens), 8, d, dtype), window=window, sinks=sinks)


def test_reference_of_the_tolerances_is_finite():
    """(A window's reference has a bound wherever it has a value.)"""
    cache = make_cache([900], [0], 1, 64, 16, torch.float16, seed=1)
    o, lse, tol, lse_tol = ref.attend(queries(3, 4, 64, torch.float16), cache.k_pages, cache.v_pages, cache.page_table, [900], [0, 3], 0.125, 40, 2)
    assert tol.isfinite().all() and lse_tol.isfinite().all() and not math.isnan(float(o.sum() + lse.sum()))
