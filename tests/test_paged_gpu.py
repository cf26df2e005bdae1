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


# --- attention -------------------------------------------------------------------------------------------------------

def queries(rows, hq, d, dtype, seed=7):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((rows, hq, d), generator=g, device=DEV).to(dtype)


def check(got, want):
    o, lse = got
    ro, rlse, tol, lse_tol = want
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    own = ~rlse.isnan()
    none = own & (rlse == -math.inf)
    assert (lse[none] == -math.inf).all() and not o[none].any()
    some = own & ~none
    assert ((lse.double() - rlse).abs() <= lse_tol)[some].all(), (lse.double() - rlse).abs()[some].max()
    bad = ~((o.double() - ro).abs() <= tol)[some]
    assert not bad.any(), (int(bad.sum()), ((o.double() - ro).abs() / tol)[some].max())


def attend(cache, q, starts=None, scale=None, window=None, sinks=0, max_new=None, max_len=None):
    """The call with outputs that hold a mark, and its reference."""
    out, lse = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
    s = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV)
    got = cache.attend(q, s, scale, window, sinks, max_new, max_len, out, lse)
    assert got[0] is out and got[1] is lse
    want = ref.attend(q, cache.k_pages, cache.v_pages, cache.page_table, cache.length.tolist(), starts,
                      cache.D ** -0.5 if scale is None else scale, window, sinks, max_len, max_new)
    check(got, want)
    left = want[1].isnan()
    assert (out[left] == 7.0).all() and (lse[left] == 7.0).all()
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_token_pages(page, d, dtype):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 701]
    cache = make_cache(lens, [0] * len(lens), 2, d, page, dtype, seed=page)
    attend(cache, queries(len(lens), 8, d, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (7, 1), (16, 2), (9, 1), (24, 2), (16, 1), (17, 1), (40, 1), (128, 1)])
def test_token_groups(hq, hkv, d, dtype):
    """One launch (short) and shares with a merge (long); groups that fill no block, one and several."""
    for lens in ([70, 1, 300], [3000, 0, 17, 2500]):
        cache = make_cache(lens, [0] * len(lens), hkv, d, 32, dtype, seed=hq)
        attend(cache, queries(len(lens), hq, d, dtype), scale=0.2)


@pytest.mark.parametrize("d", [64, 128])
def test_token_many_sequences(d):
    """More rows than SMs, lengths of every kind: rows within a share, cut by one end, cut by several."""
    lens = [(i * 37) % 900 for i in range(200)] + [20000, 0, 0, 5, 9000]
    cache = make_cache(lens, [0] * len(lens), 2, d, 64, torch.bfloat16, seed=3)
    attend(cache, queries(len(lens), 8, d, torch.bfloat16))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (63, 2), (64, 4), (65, 64), (100, 65), (1000, 4), (5000, 300), (1 << 30, 7),
                                          ((1 << 31) - 1, (1 << 31) - 1)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (64, 256)])
def test_token_window(d, page, window, sinks):
    lens = [0, 1, 16, 64, 65, 130, 700, 1064, 1065, 6000]
    cache = make_cache(lens, [0] * len(lens), 2, d, page, torch.bfloat16, seed=window % 1000)
    attend(cache, queries(len(lens), 8, d, torch.bfloat16), window=window, sinks=sinks)


def test_token_pages_out_of_the_window_are_not_read():
    """The table's places that no token sees name no page, pages of them hold NaN: nothing of it shows."""
    for page, window, sinks in ((16, 100, 5), (64, 200, 0), (256, 300, 1)):
        lens = [1000, 3000]
        cache = make_cache(lens, [0, 0], 2, 64, page, torch.bfloat16, seed=1)
        q = queries(2, 8, 64, torch.bfloat16)
        want = cache.attend(q, window=window, sinks=sinks)
        for b, n in enumerate(lens):
            lo = n - window
            for x in range(-(-n // page)):
                if x * page >= sinks and (x + 1) * page <= lo:
                    p = int(cache.page_table[b, x])
                    cache.k_pages[p], cache.v_pages[p] = math.nan, math.inf
                    cache.page_table[b, x] = (-1, 1 << 30, -(1 << 31))[x % 3]
        got = cache.attend(q, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert attn.attn_fwd_debug_status() == attn.ATTN_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_missing_pages_read_as_zeros_and_are_reported():
    for lens in ([200, 90], [5000, 90]):
        cache = make_cache(lens, [0, 0], 2, 64, 16, torch.bfloat16, seed=2)
        cache.page_table[0, 3], cache.page_table[0, 5], cache.page_table[0, 7], cache.page_table[1, 0] = -1, cache.n_pages, -(1 << 31), (1 << 31) - 1
        q = queries(2, 4, 64, torch.bfloat16)
        got = cache.attend(q)
        torch.cuda.synchronize()
        assert attn.attn_fwd_debug_status() == attn.ATTN_ERR_PAGE and attn.attn_fwd_debug_status() == attn.ATTN_OK
        check(got, ref.attend(q, cache.k_pages, cache.v_pages, cache.page_table, lens, None, 0.125))


def test_lengths_are_clamped():
    cache = make_cache([100, 400, 30], [0, 0, 0], 2, 64, 16, torch.bfloat16, seed=5)
    cap = cache.max_pages * 16
    q = queries(3, 4, 64, torch.bfloat16)
    attend(cache, q, max_len=50)
    cache.length[0] = -4
    attend(cache, q, max_len=200)
    attend(cache, q, max_len=0)
    cache.page_table[:] = 0
    cache.length[1] = cap + 1000
    cache.k_pages.nan_to_num_(0.5)
    cache.v_pages.nan_to_num_(0.5)
    attend(cache, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (5, 1), (14, 2), (100, 1)])
def test_few_tokens(hq, hkv, d, dtype):
    """Two to five new tokens of some sequences, one or none of others."""
    new, had = [3, 0, 1, 5, 2, 4], [0, 10, 700, 63, 1500, 12]
    cache = make_cache([a + b for a, b in zip(had, new)], [0] * 6, hkv, d, 16, dtype, seed=hq)
    starts, _ = starts_of(new)
    q = queries(starts[-1] + 2, hq, d, dtype)
    attend(cache, q, starts, max_new=5)
    attend(cache, q, starts, window=40, sinks=3, max_new=5)
    attend(cache, q, starts, max_new=3)


CHUNKS = [([1], [0]), ([40], [0]), ([128], [0]), ([200], [77]), ([1, 64, 0, 300], [500, 0, 9, 1]), ([257, 3, 90], [1000, 2000, 17]),
          ([700], [3000])]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,had", CHUNKS, ids=str)
def test_chunks(new, had, d, page):
    cache = make_cache([a + b for a, b in zip(had, new)], [0] * len(new), 2, d, page, torch.bfloat16, seed=d)
    starts, _ = starts_of(new)
    q = queries(starts[-1] + 5, 8, d, torch.bfloat16)
    attend(cache, q, starts)
    attend(cache, q, starts, window=100, sinks=10)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (3, 1), (10, 2), (7, 1), (12, 1), (24, 2), (100, 1), (128, 1)])
def test_chunk_groups(hq, hkv, dtype):
    for d in (64, 128):
        cache = make_cache([150, 40, 333], [0] * 3, hkv, d, 32, dtype, seed=hq)
        q = queries(150 + 9 + 33, hq, d, dtype)
        attend(cache, q, [0, 150, 159, 192], scale=0.2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (50, 0), (127, 1), (128, 128), (129, 129), (300, 4), (2000, 200)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 128)])
def test_chunk_window(d, page, window, sinks):
    new, had = [300, 1, 40, 700], [900, 200, 0, 100]
    cache = make_cache([a + b for a, b in zip(had, new)], [0] * 4, 2, d, page, torch.bfloat16, seed=window)
    starts, _ = starts_of(new)
    attend(cache, queries(starts[-1], 8, d, torch.bfloat16), starts, window=window, sinks=sinks)


def test_chunk_pages_out_of_the_window_are_not_read():
    for page, window, sinks in ((16, 100, 5), (128, 200, 0)):
        new, n = 150, 3000
        cache = make_cache([n], [0], 2, 64, page, torch.bfloat16, seed=1)
        q, s = queries(new, 8, 64, torch.bfloat16), torch.tensor([0, new], dtype=torch.int32, device=DEV)
        want = cache.attend(q, s, window=window, sinks=sinks)
        for x in range(-(-n // page)):
            if x * page >= sinks and (x + 1) * page <= n - new + 1 - window:
                p = int(cache.page_table[0, x])
                cache.k_pages[p], cache.v_pages[p] = math.nan, math.inf
                cache.page_table[0, x] = (-1, 1 << 30, -(1 << 31))[x % 3]
        got = cache.attend(q, s, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert attn.attn_fwd_debug_status() == attn.ATTN_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_tokens_than_entries():
    """Tokens before a sequence's first entry see nothing: 0 and -inf."""
    cache = make_cache([3, 0, 70], [0] * 3, 2, 64, 16, torch.bfloat16, seed=4)
    for new in ([5, 2, 70], [100, 90, 200]):
        starts, _ = starts_of(new)
        q = queries(starts[-1], 4, 64, torch.bfloat16)
        attend(cache, q, starts)
        attend(cache, q, starts, window=2, sinks=1)
    q = queries(7, 4, 64, torch.bfloat16)
    attend(cache, q, [0, 5, 7, 7], max_new=5)


def test_starts_out_of_range_and_rows_left_out():
    cache = make_cache([300, 200], [0, 0], 2, 64, 32, torch.bfloat16, seed=6)
    q = queries(64, 4, 64, torch.bfloat16)
    attend(cache, q, [-5, 20, 2000])
    attend(cache, q, [10, 40, 45])
    attend(cache, q, [10, 40, 45], max_new=20)


def test_starts_that_overlap_stay_within_the_buffers():
    """Disordered starts leave their sequences' rows undefined, and nothing else touched."""
    cache = make_cache([3000] * 6, [0] * 6, 2, 64, 32, torch.bfloat16, seed=6)
    q = queries(400, 8, 64, torch.bfloat16)
    for starts, new in (([0, 390, 0, 390, 0, 390, 0], 390), ([0, 4, 0, 4, 0, 4, 0], 2), ([390, 5, 390, -7, 390, 1 << 30, 0], 400)):
        out, lse = torch.full((404, 8, 64), 7.0, dtype=q.dtype, device=DEV), torch.full((404, 8), 7.0, device=DEV)
        s = torch.tensor(starts, dtype=torch.int32, device=DEV)
        cache.attend(q, s, max_new=new, out=out[:400], lse=lse[:400])
        cache.attend(q, s, max_new=new, max_len=500, out=out[:400], lse=lse[:400])
        torch.cuda.synchronize()
        assert attn.attn_fwd_debug_status() == attn.ATTN_OK
        assert (out[400:] == 7.0).all() and (lse[400:] == 7.0).all()


def test_more_sequences_than_the_list_takes_at_once():
    """More than 1024 sequences of a few tokens."""
    new = [(i * 7) % 5 for i in range(1500)]
    had = [(i * 13) % 70 for i in range(1500)]
    had[700] = 5000
    cache = make_cache([a + b for a, b in zip(had, new)], [0] * 1500, 1, 64, 16, torch.bfloat16, seed=6)
    starts, _ = starts_of(new)
    q = queries(starts[-1], 8, 64, torch.bfloat16)
    attend(cache, q, starts, max_new=4)
    attend(cache, q, starts, window=20, sinks=1)


def test_large_logits():
    """Logits that grow along the keys: the reference moves many times."""
    for new in (1, 200):
        cache = make_cache([2500], [0], 2, 64, 64, torch.bfloat16, seed=9)
        for x, p in enumerate(cache.page_table[0, :40].tolist()):
            cache.k_pages[p] *= 0.1 + 0.3 * x
        q = queries(new, 4, 64, torch.bfloat16)
        attend(cache, q, [0, new], scale=0.5)


def test_low_values_keep_their_bits_in_fp16():
    """The largest key's V is 0; what is left comes from keys many nats below."""
    for new in (1, 130):
        cache = make_cache([1500], [0], 1, 64, 64, torch.float16, seed=3)
        cache.k_pages.zero_()
        q = torch.zeros((new, 4, 64), dtype=torch.float16, device=DEV)
        q[..., 0] = 1.0
        p0 = int(cache.page_table[0, 0])
        cache.k_pages[p0, 0, 0, 0], cache.v_pages[p0, 0, 0] = 16.0, 0.0
        attend(cache, q, [0, new], scale=1.0)


@pytest.mark.parametrize("new", [1, 4, 150])
def test_streams_graphs_and_repeats(new):
    lens = [3000, 200, 1024]
    cache = make_cache([n + new for n in lens], [0] * 3, 2, 128, 64, torch.bfloat16, seed=8)
    starts, s = starts_of([new] * 3)
    q = queries(3 * new, 8, 128, torch.bfloat16)
    want = cache.attend(q, s, max_new=new)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = cache.attend(q, s, max_new=new, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cache.attend(q, s, max_new=new)
    cache.length -= 5  # a graph takes the lengths as they are when it runs
    graph.replay()
    torch.cuda.synchronize()
    later = cache.attend(q, s, max_new=new)
    assert torch.equal(held[0], later[0]) and torch.equal(held[1], later[1]) and not torch.equal(held[0], want[0])


def test_exchanged_buffers_and_copies():
    cache = make_cache([100, 50], [0, 0], 2, 64, 16, torch.bfloat16)
    q = queries(2, 4, 64, torch.bfloat16)
    want = cache.attend(q)
    for other in (copy.copy(cache), copy.deepcopy(cache)):
        got = other.attend(q)
        assert torch.equal(got[0], want[0])
    other = copy.deepcopy(cache)
    other.length = torch.tensor([60, 50], dtype=torch.int32, device=DEV)
    got = other.attend(q)
    assert not torch.equal(got[0], want[0]) and torch.equal(got[0][1], want[0][1])
    for name, bad in (("length", cache.length.long()), ("page_table", cache.page_table[:1]), ("k_pages", cache.k_pages.half()),
                      ("v_pages", None), ("B", 7), ("other", 1)):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            setattr(cache, name, bad)


def test_python_refusals_on_the_device():
    cache = make_cache([100, 50], [0, 0], 2, 64, 16, torch.bfloat16)
    q = queries(2, 4, 64, torch.bfloat16)
    for bad in (dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(seq_start=torch.zeros(4, dtype=torch.int32, device=DEV)),
                dict(window=0), dict(out=q.float()), dict(lse=torch.zeros(4, 2, device=DEV))):
        with pytest.raises(ValueError):
            cache.attend(**{**dict(q=q), **bad})
    with pytest.raises(TypeError):
        cache.attend(q.half())
    for bad in (dict(sinks=-1), dict(max_len=1 << 20), dict(scale=0.0), dict(max_len=1 << 33), dict(window=1 << 33)):
        with pytest.raises(attn.AttnError):
            cache.attend(q, **bad)
    k = queries(2, 2, 64, torch.bfloat16)
    for bad in (dict(k=k[:1]), dict(v=k[:, :1]), dict(q=q[:1]), dict(q_out=q), dict(q_weight=k[0, 0]), dict(q=q, q_out=q[:1]),
                dict(length_out=cache.length.long())):
        with pytest.raises(ValueError):
            cache.append(**{**dict(k=k, v=k), **bad})
    with pytest.raises(TypeError):
        cache.append(k.half(), k.half())
    with pytest.raises(ValueError):
        attn.PagedKVCache.empty(1, 1, 4, 24, 2, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_conversation(dtype):
    """A prompt, tokens, another message and tokens again, normed and turned on the way, against one pass over it all in 64 bits."""
    H, G, d, page = 2, 4, 64, 16
    f = attn.rotary_frequencies(d)
    rope = attn.Rotary(f)
    g = torch.Generator(device=DEV).manual_seed(2)
    w = list((1 + 0.2 * torch.randn((2, d), generator=g, device=DEV)).to(dtype))
    steps = [[37, 90, 1], [1, 1, 1], [1, 1, 1], [60, 1, 5], [1, 1, 1]]
    total = [sum(s[b] for s in steps) for b in range(3)]
    cache = make_cache([0, 0, 0], total, H, d, page, dtype)
    rows = [[], [], []]
    for step in steps:
        starts, s = starts_of(step)
        qkv = torch.randn((starts[-1], H * (G + 2), d), generator=g, device=DEV).to(dtype)
        q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
        q = cache.append(k, v, seq_start=s, q=q, rope=rope, q_weight=w[0], k_weight=w[1])
        o, lse = cache.attend(q, s, window=50, sinks=2, max_new=max(step))
        for b in range(3):
            rows[b].append((q[starts[b]:starts[b + 1]], k[starts[b]:starts[b + 1]], v[starts[b]:starts[b + 1]], o[starts[b]:starts[b + 1]]))
        check((o, lse), ref.attend(q, cache.k_pages, cache.v_pages, cache.page_table, cache.length.tolist(), starts, d ** -0.5, 50, 2))
    assert cache.length.tolist() == total
    for b in range(3):
        k = torch.cat([r[1] for r in rows[b]])
        want, tol = ref.forward(k, w[1], torch.arange(total[b], device=DEV), f, False, 1.0, 1e-6)
        kk, vv = rows_of(cache, b, 0, total[b])
        assert ((kk.double() - want).abs() <= tol).all() and torch.equal(vv, torch.cat([r[2] for r in rows[b]]))


@pytest.mark.parametrize("new,hq", [(1, 8), (1, 16), (40, 8), (300, 8)])
def test_back_to_back(new, hq):
    """Many calls without a wait between them, over more tiles than the rings hold: the same each time."""
    cache = make_cache([6000 + new] * 4, [0] * 4, 4 if hq == 16 else 2, 128, 64, torch.bfloat16, seed=new)
    if hq == 16:
        hq = 64  # 16 query heads a key head: two tiles of 8 rows
    starts, s = starts_of([new] * 4)
    q = queries(4 * new, hq, 128, torch.bfloat16)
    first = attend(cache, q, starts, max_new=new)
    got = [cache.attend(q, s, max_new=new) for _ in range(30)]
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    for o, lse in got:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("new", [1, 40])
def test_queries_of_any_row_stride(new):
    """q as slices of a fused projection's rows, lengths that differ."""
    cache = make_cache([700, 30 + new], [0, 0], 2, 128, 32, torch.bfloat16, seed=new)
    starts, s = starts_of([new, new])
    wide = queries(2 * new, 12, 128, torch.bfloat16)
    q = wide[:, 2:10]
    a, b = attend(cache, q, starts, max_new=new), attend(cache, q.contiguous(), starts, max_new=new)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(attn.AttnError):
        cache.attend(q[:1].expand(2 * new, 8, 128), s, max_new=new)
    with pytest.raises(ValueError):
        cache.attend(wide[:, ::2], s, max_new=new)


def test_places_beyond_32_bits():
    """Pages whose elements, and queries whose rows, lie behind 2^32 and 2^31 of their buffers."""
    H, page, d = 8, 256, 128
    n_pages = (1 << 32) // (H * page * d) + 40
    cache = attn.PagedKVCache.empty(2, H, n_pages, page, 5, d)  # 8.6 GB each of K and V
    last = torch.arange(n_pages - 10, n_pages, dtype=torch.int32, device=DEV)
    cache.page_table.copy_(last.flip(0).view(2, 5))
    rows = (1 << 31) // (32 * d) + 600
    g = torch.Generator(device=DEV).manual_seed(3)
    new = [1100, 250]
    at, s = starts_of(new)
    k, v = torch.randn((2, at[-1], H, d), generator=g, device=DEV).bfloat16()
    cache.append(k, v, seq_start=s)
    for b in range(2):
        kk, vv = rows_of(cache, b, 0, new[b])
        assert torch.equal(kk, k[at[b]:at[b + 1]]) and torch.equal(vv, v[at[b]:at[b + 1]])
    first = rows - 250  # the queries are the last rows of 4.3 GB
    big = torch.empty((rows, 32, d), dtype=torch.bfloat16, device=DEV)
    big[first:] = torch.randn((250, 32, d), generator=g, device=DEV).bfloat16()
    out, lse = torch.empty_like(big), torch.empty((rows, 32), device=DEV)
    for n in ([1, 2], [50, 200]):
        e = first + sum(n)
        starts = torch.tensor([first, first + n[0], e], dtype=torch.int32, device=DEV)
        cache.attend(big, starts, max_new=max(n), out=out, lse=lse)
        check((out[first:e], lse[first:e]), ref.attend(big[first:e], cache.k_pages[n_pages - 10:], cache.v_pages[n_pages - 10:],
                                                       cache.page_table - (n_pages - 10), new, [0, n[0], sum(n)], d ** -0.5))


def test_decoding_steps_in_one_graph():
    """A step's append and attention, captured once: lengths grow in place with each replay."""
    had, H, d = [37, 0, 300], 2, 64
    cache = make_cache(had, [8] * 3, H, d, 16, torch.bfloat16, seed=5)
    twin = copy.deepcopy(cache)
    rope = attn.Rotary(attn.rotary_frequencies(d))
    qkv = torch.empty((3, 8 + 2 * H, d), dtype=torch.bfloat16, device=DEV)

    def step(c):
        q = c.append(qkv[:, 8:8 + H], qkv[:, 8 + H:], q=qkv[:, :8], rope=rope)
        return c.attend(q, max_len=310)

    g = torch.Generator(device=DEV).manual_seed(6)
    qkv.normal_(generator=g)
    warm = copy.deepcopy(cache)
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(cache)
    for i in range(5):
        qkv.normal_(generator=g)
        graph.replay()
        want = step(twin)
        torch.cuda.synchronize()
        assert cache.length.tolist() == [n + i + 1 for n in had]
        assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK


@pytest.mark.parametrize("B,turns", [(3, 40), (300, 6)])
def test_old_and_new_lengths_side_by_side(B, turns):
    """Two rows of one buffer in turn, and a piece of a longer one in place, against buffers of their own."""
    H, d, page = 2, 64, 16
    apart = attn.PagedKVCache.empty(B, H, B * 4, page, 4, d)
    apart.page_table.copy_(torch.arange(B * 4, dtype=torch.int32, device=DEV).view(B, 4))
    pair = torch.zeros((2, B), dtype=torch.int32, device=DEV)
    piece = torch.full((B + 7,), 9, dtype=torch.int32, device=DEV)
    turned, inside = (attn.PagedKVCache(torch.empty_like(apart.k_pages), torch.empty_like(apart.v_pages), apart.page_table, x)
                      for x in (pair[0], piece[5:5 + B]))
    turned.length.zero_(), inside.length.zero_()
    g = torch.Generator(device=DEV).manual_seed(9)
    qkv = torch.randn((turns, B, 4 + 2 * H, d), generator=g, device=DEV).bfloat16()
    rope = attn.Rotary(attn.rotary_frequencies(d))
    got = []
    for c in (apart, turned, inside):
        steps = []
        for i in range(turns):
            out = pair[1 - i % 2] if c is turned else None
            q = c.append(qkv[i, :, 4:4 + H], qkv[i, :, 4 + H:], q=qkv[i, :, :4], rope=rope, length_out=out)
            if c is turned:
                c.length = out
            steps.append(c.attend(q))
        got.append(steps)
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    assert (piece[:5] == 9).all() and (piece[5 + B:] == 9).all() and (piece[5:5 + B] == turns).all() and (turned.length == turns).all()
    for steps in got[1:]:
        for x, y in zip(steps, got[0]):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_calls_on_two_streams_at_once():
    """Reads of one cache side by side, each with a workspace of its own."""
    cache = make_cache([5000, 3000], [0, 0], 2, 128, 64, torch.bfloat16, seed=7)
    s = torch.tensor([0, 60, 100], dtype=torch.int32, device=DEV)
    q1, q2 = queries(2, 8, 128, torch.bfloat16, 1), queries(100, 8, 128, torch.bfloat16, 2)
    want = cache.attend(q1), cache.attend(q2, s, max_new=60)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((cache.attend(q1, stream=streams[0]), cache.attend(q2, s, max_new=60, stream=streams[1])))
    torch.cuda.synchronize()
    for pair in got:
        for (o, lse), (wo, wl) in zip(pair, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
