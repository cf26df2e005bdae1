"""The paged K/V cache against the 64-bit definition."""
from __future__ import annotations

import copy
import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import rotary_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make_cache(lens, room, H, d, page, dtype, seed=0, fill=math.nan, spare=3):
    """A cache whose sequences hold `lens` entries and have pages for `room` more each; rows that hold none are `fill`."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-(n + r) // page) for n, r in zip(lens, room)]
    n_pages = sum(need) + spare
    cache = attn.PagedKVCache.empty(len(lens), H, n_pages, page, max(1, max(need)) + 1, d, dtype)
    cache.k_pages.fill_(fill)
    cache.v_pages.fill_(fill)
    order = torch.randperm(n_pages, generator=g, device=DEV).int()
    at = 0
    for b, (n, x) in enumerate(zip(lens, need)):
        cache.page_table[b, :x] = order[at:at + x]
        at += x
        j = torch.arange(n, device=DEV)
        where = cache.page_table[b].long()[j // page]
        for pages in (cache.k_pages, cache.v_pages):
            pages[where, :, j % page] = torch.randn((n, H, d), generator=g, device=DEV).to(dtype)
    cache.length.copy_(torch.tensor(lens, dtype=torch.int32))
    return cache


def starts_of(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at, torch.tensor(at, dtype=torch.int32, device=DEV)


def rows_of(cache, b, first, n):
    """Entries first .. first + n - 1 of sequence b."""
    j = torch.arange(first, first + n, device=DEV)
    where = cache.page_table[b].long()[j // cache.page]
    return cache.k_pages[where, :, j % cache.page], cache.v_pages[where, :, j % cache.page]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,rot,inter,weights", [(64, 64, False, True), (64, 32, True, False), (128, 128, False, True), (128, 96, True, True),
                                                 (128, 0, False, False)])
def test_append(d, rot, inter, weights, page, dtype):
    had, new, pad = [0, 5, 100, 255, 300, 17], [3, 0, 60, 1, 290, 16], 4
    cache = make_cache(had, new, 2, d, page, dtype, seed=page)
    g = torch.Generator(device=DEV).manual_seed(1)
    at, s = starts_of(new)
    qkv = torch.randn((at[-1] + pad, 6 + 4, d), generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    w = list((1 + 0.3 * torch.randn((2, d), generator=g, device=DEV)).to(dtype)) if weights else [None, None]
    f = attn.rotary_frequencies(rot) if rot else []
    rope = attn.Rotary(f, interleaved=inter, amplitude=1.1) if rot else None
    before = [x.clone() for x in (cache.k_pages, cache.v_pages)]
    q_out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    got = cache.append(k, v, seq_start=s, q=q, rope=rope, q_weight=w[0], k_weight=w[1], q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out and attn.attn_fwd_debug_status() == attn.ATTN_OK
    assert cache.length.tolist() == [a + b for a, b in zip(had, new)]
    assert (q_out[at[-1]:] == 7.0).all()
    for b, (n, m) in enumerate(zip(had, new)):
        r = slice(at[b], at[b + 1])
        pos = torch.arange(n, n + m, device=DEV)
        kk, vv = rows_of(cache, b, n, m)
        assert torch.equal(vv, v[r])
        for x, y, ww in ((q[r], q_out[r], w[0]), (k[r], kk, w[1])):
            want, tol = ref.forward(x, ww, pos, f, inter, 1.1, 1e-6)
            assert ((y.double() - want).abs() <= tol).all()
        # put back, nothing else has changed
        j = torch.arange(n, n + m, device=DEV)
        where = cache.page_table[b].long()[j // page]
        for x, y in zip((cache.k_pages, cache.v_pages), before):
            x[where, :, j % page] = y[where, :, j % page]
    for x, y in zip((cache.k_pages, cache.v_pages), before):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_append_a_token_each_and_length_out():
    had = [0, 15, 16, 255, 1000]
    cache = make_cache(had, [1] * 5, 4, 64, 16, torch.bfloat16)
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v = torch.randn((2, 5, 4, 64), generator=g, device=DEV).bfloat16()
    out = torch.full((5,), -7, dtype=torch.int32, device=DEV)
    assert cache.append(k, v, length_out=out) is None
    torch.cuda.synchronize()
    assert out.tolist() == [n + 1 for n in had] and cache.length.tolist() == had
    for b, n in enumerate(had):
        kk, vv = rows_of(cache, b, n, 1)
        assert torch.equal(kk[0], k[b]) and torch.equal(vv[0], v[b])


def test_append_beyond_the_capacity_and_without_a_page():
    cache = make_cache([30, 10, 0], [2, 40, 40], 2, 64, 16, torch.bfloat16, fill=0.0)
    cache.page_table[0, 2:] = -1
    cap = cache.max_pages * 16
    cache.length[0] = cap - 2           # two entries of four fit, on no page
    cache.page_table[1, 1] = cache.n_pages  # entries 16 .. 31 of the second have none
    before = [x.clone() for x in (cache.k_pages, cache.v_pages)]
    at, s = starts_of([4, 12, 1])
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = torch.randn((2, 17, 2, 64), generator=g, device=DEV).bfloat16()
    q = torch.randn((17, 2, 64), generator=g, device=DEV).bfloat16()
    rope = attn.Rotary(attn.rotary_frequencies(64))
    q_out = cache.append(k, v, seq_start=s, q=q, rope=rope)
    torch.cuda.synchronize()
    # both failures, one reading each
    assert [attn.attn_fwd_debug_status() for _ in range(3)] == [attn.ATTN_ERR_CAPACITY, attn.ATTN_ERR_PAGE, attn.ATTN_OK]
    assert cache.length.tolist() == [cap, 22, 1]
    pos = torch.tensor([cap - 2, cap - 1, cap, cap + 1, *range(10, 22), 0], device=DEV)
    want, tol = ref.forward(q, None, pos, attn.rotary_frequencies(64), False, 1.0, 1e-6)
    assert ((q_out.double() - want).abs() <= tol).all()
    # six rows of the second sequence and the third's one have been written, nothing else
    p1, p2 = int(cache.page_table[1, 0]), int(cache.page_table[2, 0])
    assert torch.equal(cache.v_pages[p1, :, 10:].transpose(0, 1), v[4:10]) and torch.equal(cache.v_pages[p2, :, 0], v[16])
    for x, y in zip((cache.k_pages, cache.v_pages), before):
        x[p1, :, 10:], x[p2, :, 0] = y[p1, :, 10:], y[p2, :, 0]
        assert torch.equal(x, y)


def test_append_lengths_and_starts_out_of_range():
    """A negative length counts as 0, starts outside the rows as their ends."""
    cache = make_cache([0, 0], [40, 40], 2, 64, 16, torch.bfloat16, fill=0.0)
    cache.length[0] = -9
    s = torch.tensor([-3, 10, 500], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    k, v = torch.randn((2, 30, 2, 64), generator=g, device=DEV).bfloat16()
    cache.append(k, v, seq_start=s)
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK and cache.length.tolist() == [10, 20]
    for b, (a, e) in enumerate(((0, 10), (10, 30))):
        kk, vv = rows_of(cache, b, 0, e - a)
        assert torch.equal(kk, k[a:e]) and torch.equal(vv, v[a:e])


def test_append_no_rows():
    cache = make_cache([7, 3], [1, 1], 2, 64, 16, torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.full((2,), -1, dtype=torch.int32, device=DEV)
    cache.append(e, e, seq_start=s, length_out=out)
    cache.append(e, e, seq_start=s)
    torch.cuda.synchronize()
    assert out.tolist() == [7, 3] and cache.length.tolist() == [7, 3]
