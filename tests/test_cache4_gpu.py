"""The 4-bit K/V cache: append, read, attention of one token, eviction, and a
run of them together, against the 64-bit definitions."""
from __future__ import annotations

import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def starts_of(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def filled(B, H, cap, D, lens, seed=0, poison=True):
    """A cache of random entries; what lies behind the lengths is poison."""
    g = gen(seed)
    c = attn.KVCache4.empty(B, H, cap, D)
    x = torch.randn((2, B, H, cap, D), generator=g, device="cuda")
    x[0, ..., 3::17] += 4.0
    for codes, meta, y in ((c.k_codes, c.k_meta, x[0]), (c.v_codes, c.v_meta, x[1])):
        code, s, m = ref.quantise(y.bfloat16())
        codes.copy_(ref.pack(code))
        meta.copy_(torch.stack([s, m], -1))
    c.weight.copy_(torch.rand((B, H, cap), generator=g, device="cuda"))
    c.pos.copy_(torch.arange(cap, device="cuda").expand(B, H, cap))
    c.length.copy_(torch.tensor(lens, dtype=torch.int32))
    if poison:
        for b, n in enumerate(lens):
            n = max(n, 0)
            c.k_codes[b, :, n:] = 255
            c.v_codes[b, :, n:] = 255
            c.k_meta[b, :, n:] = math.nan
            c.v_meta[b, :, n:] = math.inf
            c.weight[b, :, n:] = math.nan
            c.pos[b, :, n:] = 1 << 30
    return c


def ok():
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK


# --- append and read -------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128), (8, 128), (5, 64)])
@pytest.mark.parametrize("lens,start", [([1], [0]), ([3, 0, 17], [5, 2, 0]), ([33, 1, 0, 64, 7], [0, 63, 9, 1, 2])], ids=str)
def test_append(H, D, lens, start, dtype):
    cap, rows = 100, sum(lens) + 6
    c = filled(len(lens), H, cap, D, start)
    before = [x.clone() for x in (c.k_codes, c.k_meta, c.v_codes, c.v_meta, c.weight, c.pos)]
    kv = (3 * torch.randn((rows, 2 * H, D), generator=gen(3), device="cuda")).to(dtype)
    kv[0, 0] = 1.5  # a constant row: s = 0
    kv[1, H:] *= 1e-30 if dtype == torch.bfloat16 else 1e-4
    k, v = kv[:, :H], kv[:, H:]
    first = torch.arange(len(lens), dtype=torch.int32, device="cuda") * 1000
    out = torch.empty_like(c.length)
    c.append(k, v, seq_start=starts_of(lens), first_pos=first, length_out=out)
    ok()
    assert c.length.tolist() == start and out.tolist() == [a + b for a, b in zip(lens, start)]
    at = 0
    for b, n in enumerate(lens):
        for x, codes, meta, i in ((k, c.k_codes, c.k_meta, 0), (v, c.v_codes, c.v_meta, 2)):
            code, s, m = ref.quantise(x[at:at + n].transpose(0, 1))
            before[i][b, :, start[b]:start[b] + n] = ref.pack(code)
            before[i + 1][b, :, start[b]:start[b] + n] = torch.stack([s, m], -1).bfloat16()
        before[4][b, :, start[b]:start[b] + n] = 0
        before[5][b, :, start[b]:start[b] + n] = torch.arange(n, device="cuda", dtype=torch.int32) + 1000 * b
        at += n
    for got, want, name in zip((c.k_codes, c.k_meta, c.v_codes, c.v_meta, c.weight, c.pos), before, ("k", "km", "v", "vm", "w", "p")):
        assert torch.equal(got.view(torch.int16) if got.dtype == torch.bfloat16 else got.nan_to_num(-1.0) if got.is_floating_point() else got,
                           want.view(torch.int16) if want.dtype == torch.bfloat16 else want.nan_to_num(-1.0) if want.is_floating_point() else want), name


def test_append_rounding_is_the_formats():
    """Values on and next to the half way points, in fp32 divisions against 64-bit ones: the codes are equal, all of them."""
    g = gen(7)
    x = torch.randn((4096, 2, 128), generator=g, device="cuda").bfloat16()
    x[:, :, 0], x[:, :, 1] = 0.0, 15.0  # s = 1, m = 0 ...
    x[:, :, 2:64] = (torch.randint(0, 31, (4096, 2, 62), generator=g, device="cuda") / 2).bfloat16()  # ... and halves
    x[:, :, 64:] *= torch.logspace(-20, 20, 4096, device="cuda").bfloat16()[:, None, None]
    c = attn.KVCache4.empty(1, 2, 4096, 128)
    c.append(x, x, seq_start=starts_of([4096]))
    ok()
    code, s, m = ref.quantise(x.transpose(0, 1))
    assert torch.equal(c.k_meta[0].double(), torch.stack([s, m], -1))
    # a 64-bit division may fall on the other side of a half way point that the 32-bit one lands on: such values lie
    # within 2^-23 relative of it, and only those may differ, by one
    got, want = ref.unpack(c.k_codes[0]), code
    q = ((x.transpose(0, 1).double().unflatten(-1, (-1, 64)) - m[..., None]) / s[..., None]).flatten(-2)
    near = ((q - q.floor() - 0.5).abs() <= 16 * 2.0 ** -23)
    assert torch.equal(got[~near], want[~near]) and ((got - want).abs()[near] <= 1).all()
    assert torch.equal(got[..., :64], want[..., :64])  # exact halves go to the even code


def test_append_single_tokens_in_place_and_beyond_the_capacity():
    c = filled(3, 2, 10, 64, [0, 9, 10])
    k = torch.randn((3, 2, 64), generator=gen(1), device="cuda").bfloat16()
    full = c.k_codes[2].clone()
    c.append(k, k)
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_ERR_CAPACITY
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK  # read and cleared
    assert c.length.tolist() == [1, 10, 10]
    assert c.pos[0, :, 0].tolist() == [0, 0] and c.pos[1, :, 9].tolist() == [9, 9]
    assert torch.equal(c.k_codes[2], full)
    rows = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    back, _ = c.read(first_slot=torch.cat([rows, rows[:1]]), dtype=torch.float32)
    code, s, m = ref.quantise(k[:2])
    assert torch.equal(back[:2].double(), ref.values(ref.pack(code), torch.stack([s, m], -1)))


def test_append_counts_only_rows_there_are():
    """Starts before the first row and behind the last, and a negative length: entries are as many as rows."""
    k = torch.randn((10, 2, 64), generator=gen(1), device="cuda").bfloat16()
    for in_place in (False, True):
        c = filled(3, 2, 50, 64, [4, 7, 0])
        c.length[2] = -3
        start = torch.tensor([-5, 3, 8, 400], dtype=torch.int32, device="cuda")
        out = c.length if in_place else torch.empty_like(c.length)
        c.append(k, k, seq_start=start, length_out=out)
        ok()
        assert out.tolist() == [7, 12, 2]
        code, s, m = ref.quantise(k)
        for b, (row, n, slot) in enumerate(((0, 3, 4), (3, 5, 7), (8, 2, 0))):
            assert torch.equal(c.k_codes[b, :, slot:slot + n], ref.pack(code[row:row + n]).transpose(0, 1))
            assert c.pos[b, 0, slot:slot + n].tolist() == list(range(slot, slot + n))


def test_not_finite_groups_stand_for_nan_alone():
    x = torch.randn((3, 1, 128), generator=gen(1), device="cuda").bfloat16()
    x[0, 0, 5], x[1, 0, 70], x[2, 0, 127] = math.nan, math.inf, -math.inf
    c = attn.KVCache4.empty(3, 1, 4, 128)
    c.append(x, torch.zeros_like(x))
    k, v = c.read(dtype=torch.float32)
    ok()
    assert k[0, 0, :64].isnan().all() and k[1, 0, 64:].isnan().all() and k[2, 0, 64:].isnan().all()
    assert k[0, 0, 64:].isfinite().all() and k[1:, 0, :64].isfinite().all() and (v == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_read(D, dtype):
    B, H, cap = 3, 2, 40
    c = filled(B, H, cap, D, [40, 40, 40], seed=2)
    want = [ref.values(c.k_codes, c.k_meta), ref.values(c.v_codes, c.v_meta)]
    first = torch.tensor([30, 0, 3], dtype=torch.int32, device="cuda")
    lens = [12, 5, 0]  # the first reaches 2 slots past the capacity
    k, v = (torch.full((20, H, D), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    got = c.read(seq_start=starts_of(lens), first_slot=first, k_out=k, v_out=v)
    ok()
    assert got[0] is k and got[1] is v
    for x, w in zip(got, want):
        assert torch.equal(x[:10], w[0, :, 30:40].transpose(0, 1).to(dtype))
        assert (x[10:12] == 9.0).all() and (x[17:] == 9.0).all()
        assert torch.equal(x[12:17], w[1, :, :5].transpose(0, 1).to(dtype))


# --- attention of one token ------------------------------------------------------------------------------------------

def check_attend(c, q, lens, scale=None, weight=True, **kw):
    D = c.D
    w_out = torch.full_like(c.weight, 5.0) if weight else None
    w_in = c.weight.clone()
    o, lse = c.attend(q, scale=scale, weight_out=w_out, **kw)
    ok()
    ro, rlse, rw, tol, lse_tol, w_tol = ref.decode(q, c, lens, scale if scale is not None else D ** -0.5)
    none = rlse == -math.inf
    assert (lse[none] == -math.inf).all() and (o[none] == 0).all()
    assert ((lse.double() - rlse).abs() <= lse_tol)[~none].all(), (lse.double() - rlse).abs()[~none].max()
    bad = (o.double() - ro).abs() > tol
    assert not bad.any(), (int(bad.sum()), ((o.double() - ro).abs() / tol.clamp(min=1e-30)).max())
    if weight:
        there = torch.arange(c.capacity, device="cuda")[None, None] < torch.tensor(lens, device="cuda").clamp(0, c.capacity)[:, None, None]
        assert (w_out[~there.expand_as(w_out)] == 5.0).all()
        # one more fp32 addition onto the weight that was there
        err = (w_out.double() - (w_in.double() + rw)).abs()
        assert (err <= w_tol + (w_in.double().abs() + rw) * 2.0 ** -24 * 2)[there.expand_as(err)].all()
    return o, lse, w_out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [0, 63, 64, 65, 0], [200, 1, 127, 128, 129], [1000]], ids=str)
def test_attend_lengths(lens, D, dtype):
    c = filled(len(lens), 2, 1000, D, lens, seed=len(lens))
    q = torch.randn((len(lens), 8, D), generator=gen(1), device="cuda").to(dtype)
    check_attend(c, q, lens)
    check_attend(c, q, lens, weight=False)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (7, 1), (8, 1), (9, 1), (16, 1), (12, 4), (40, 2), (128, 1), (20, 20)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_groups(hq, hkv, dtype):
    lens = [130, 0, 77, 300]
    for D in (64, 128):
        c = filled(4, hkv, 300, D, lens, seed=hq)
        q = torch.randn((4, hq, D), generator=gen(hq), device="cuda").to(dtype)
        check_attend(c, q, lens)


def test_attend_shares_cross_sequences():
    """More tiles than CTAs: a CTA's share runs over ends of sequences and heads, and a long row has many shares."""
    lens = [(i * 977) % 3000 for i in range(37)] + [20000]
    c = filled(38, 3, 20000, 64, lens, seed=1)
    q = torch.randn((38, 6, 64), generator=gen(1), device="cuda").bfloat16()
    check_attend(c, q, lens)


def test_attend_many_sequences():
    """More sequences than threads find the start of a share."""
    lens = [(i * 7) % 90 for i in range(700)]
    c = filled(700, 1, 90, 64, lens, seed=1)
    q = torch.randn((700, 4, 64), generator=gen(1), device="cuda").bfloat16()
    check_attend(c, q, lens)


def test_attend_max_len_and_lengths_out_of_range():
    c = filled(3, 2, 256, 128, [256, 256, 256], seed=1)
    q = torch.randn((3, 4, 128), generator=gen(1), device="cuda").bfloat16()
    c.length.copy_(torch.tensor([100000, -7, 50], dtype=torch.int32))
    check_attend(c, q, [256, 0, 50])
    o, lse = c.attend(q, max_len=70)
    ok()
    ro, rlse, _, tol, lse_tol, _ = ref.decode(q, c, [70, 0, 50], 128 ** -0.5)
    assert ((o.double() - ro).abs() <= tol).all() and ((lse - rlse).abs() <= lse_tol)[rlse > -math.inf].all()


def test_attend_strided_queries_weights_in_place_and_repeatable():
    lens = [300, 40]
    c = filled(2, 2, 300, 128, lens, seed=3)
    qkv = torch.randn((2, 12, 128), generator=gen(1), device="cuda").bfloat16()
    q = qkv[:, :8]
    a = check_attend(c, q, lens)
    before = c.weight.clone()
    o, lse = c.attend(q, weight_out=c.weight)
    ok()
    assert torch.equal(o, a[0]) and torch.equal(lse, a[1])
    for b, n in enumerate(lens):
        assert torch.equal(c.weight[b, :, :n], a[2][b, :, :n])
        assert torch.equal(c.weight[b, :, n:].isnan(), before[b, :, n:].isnan())


def test_attend_peaked_and_rising_logits():
    """One key takes nearly all the weight, and logits that rise with the slot: the reference moves tile after tile."""
    lens = [900, 900]
    c = filled(2, 1, 900, 128, lens, seed=4)
    c.k_meta[0] *= torch.linspace(0.05, 8, 900, device="cuda")[None, :, None, None].bfloat16()
    c.k_meta[1, :, 333] *= 20
    q = torch.randn((2, 8, 128), generator=gen(1), device="cuda").bfloat16()
    for dtype in (torch.bfloat16, torch.float16):
        check_attend(c, q.to(dtype), lens, scale=0.3)


def test_attend_offsets_beyond_32_bits():
    """A cache of 2^32 bytes of codes and more: the last sequence's entries lie behind 2^31 elements."""
    B, H, cap, D = 3, 8, 1 << 20, 128
    small = filled(1, H, 200, D, [200], seed=5)
    c = attn.KVCache4.empty(B, H, cap, D)
    assert c.k_codes.numel() > (1 << 30) and c.weight.numel() * D // 2 > (1 << 30)
    lens = [3, 0, 200]
    for name in ("k_codes", "k_meta", "v_codes", "v_meta", "weight", "pos"):
        getattr(c, name)[2, :, :200] = getattr(small, name)[0]
        getattr(c, name)[0, :, :3] = getattr(small, name)[0, :, :3]
    c.length.copy_(torch.tensor(lens, dtype=torch.int32))
    q = torch.randn((3, 16, D), generator=gen(1), device="cuda").bfloat16()
    o, lse = c.attend(q, weight_out=c.weight, max_len=200)
    want = small.attend(q[2:], weight_out=small.weight)
    ok()
    ro, rlse, _, tol, lse_tol, _ = ref.decode(q[2:], small, [200], D ** -0.5)
    assert ((o[2:].double() - ro).abs() <= tol).all() and ((want[0].double() - ro).abs() <= tol).all()
    assert ((lse[2:] - rlse).abs() <= lse_tol).all()
    assert torch.allclose(c.weight[2, :, :200], small.weight[0], atol=1e-6)
    x = torch.randn((3, H, D), generator=gen(2), device="cuda").bfloat16()
    c.append(x, x)
    k, _ = c.read(first_slot=torch.tensor(lens, dtype=torch.int32, device="cuda"), dtype=torch.float32)
    ok()
    code, s, m = ref.quantise(x)
    assert torch.equal(k.double(), ref.values(ref.pack(code), torch.stack([s, m], -1)))


def test_attend_nan_query_stays_with_its_head():
    c = filled(2, 2, 100, 64, [100, 100], seed=6)
    q = torch.randn((2, 8, 64), generator=gen(1), device="cuda").bfloat16()
    good = c.attend(q)
    bad = q.clone()
    bad[1, 3, 7] = math.nan
    o, lse = c.attend(bad)
    ok()
    assert o[1, 3].isnan().all() and lse[1, 3].isnan()
    keep = torch.ones((2, 8), dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.equal(o[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])


# --- eviction --------------------------------------------------------------------------------------------------------

def check_evict(c, lens, budget, recent, in_place, **kw):
    B, H = c.B, c.H_kv
    names = ("k_codes", "k_meta", "v_codes", "v_meta", "weight", "pos")
    before = {n: getattr(c, n).clone() for n in names}
    w, p = before["weight"].cpu(), before["pos"].cpu()
    if in_place:
        c.evict(budget, recent, **kw)
        after = c
    else:
        out = torch.full_like(c.weight, 5.0), torch.full_like(c.pos, 5), torch.full_like(c.length, 5)
        c.evict(budget, recent, weight_out=out[0], pos_out=out[1], length_out=out[2], **kw)
        assert c.length.tolist() == lens
        after = attn.KVCache4(c.k_codes, c.k_meta, c.v_codes, c.v_meta, *out)
    ok()
    assert after.length.tolist() == [min(n, budget) for n in lens]
    for b in range(B):
        for h in range(H):
            n = lens[b]
            src = torch.tensor(ref.evict(w[b, h, :n].tolist(), p[b, h, :n].tolist(), n, budget, recent), device="cuda", dtype=torch.long)
            left = len(src)
            for name in names:
                got, want = getattr(after, name)[b, h], before[name][b, h]
                same = torch.equal(got[:left].nan_to_num(-1.0), want[src].nan_to_num(-1.0)) if got.is_floating_point() else torch.equal(got[:left], want[src])
                assert same, (b, h, name)
                rest = got[left:]
                if name in ("weight", "pos") and not in_place:
                    assert (rest == 5).all()
                else:
                    assert torch.equal(rest.nan_to_num(-1.0), want[left:].nan_to_num(-1.0)) if rest.is_floating_point() else torch.equal(rest, want[left:])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (7, 3), (64, 0), (64, 64), (299, 10), (300, 300), (1000, 5)])
def test_evict(budget, recent, D, in_place):
    lens = [300, 0, 1, 65, 64, 257]
    c = filled(6, 2, 300, D, lens, seed=budget)
    # positions in no order, weights with many ties, zeros and odd values
    for b, n in enumerate(lens):
        for h in range(2):
            c.pos[b, h, :n] = torch.randperm(n, generator=gen(b + h), device="cuda").int() * 2
    c.weight.copy_(torch.where(c.weight.isnan(), c.weight, (c.weight * 10).floor()))
    c.weight[0, 0, :5] = torch.tensor([math.nan, -0.0, 0.0, math.inf, -1.0], device="cuda")
    check_evict(c, lens, budget, recent, in_place)


@pytest.mark.parametrize("B,H,n,budget", [(1, 1, 50000, 20000), (1, 2, 9000, 8999), (2, 1, 100000, 17), (16, 8, 1500, 700)])
def test_evict_long(B, H, n, budget):
    """Slices over a cluster of CTAs, large and small budgets."""
    lens = [n] + [n // 2] * (B - 1)
    c = filled(B, H, n, 64, lens, seed=n)
    check_evict(c, lens, budget, min(budget, 100), True)


def test_evict_longest():
    n = 8 * 48 * 1024  # a cluster's shared memory is full of keys
    c = attn.KVCache4.empty(1, 1, n, 64)
    c.weight.copy_(torch.rand((1, 1, n), generator=gen(1), device="cuda"))
    c.weight[0, 0, 1000:300000] = 0.75  # ties across the slices of several CTAs
    c.pos.copy_(torch.arange(n, device="cuda"))
    c.k_codes.copy_(torch.randint(0, 256, c.k_codes.shape, generator=gen(2), device="cuda", dtype=torch.uint8))
    c.v_codes.copy_(c.k_codes.flip(2))
    c.k_meta.zero_()
    c.v_meta.zero_()
    c.length.fill_(n)
    check_evict(c, [n], 200000, 10, True)


def test_evict_all_weights_equal_keeps_the_first_slots():
    c = filled(1, 1, 500, 64, [500])
    c.weight.zero_()
    before = c.k_codes.clone()
    c.evict(100)
    ok()
    assert torch.equal(c.k_codes, before) and c.pos[0, 0, :100].tolist() == list(range(100))


def test_evict_max_len_bounds_the_lengths():
    c = filled(1, 1, 200, 64, [200], seed=1)
    w, p = c.weight[0, 0].tolist(), c.pos[0, 0].tolist()
    k = c.k_codes.clone()
    c.evict(20, 2, max_len=90)
    ok()
    src = ref.evict(w[:90], p[:90], 90, 20, 2)
    assert c.length.tolist() == [20] and torch.equal(c.k_codes[0, 0, :20], k[0, 0, src])


# --- together --------------------------------------------------------------------------------------------------------

def test_prompt_then_tokens_in_a_bounded_cache():
    """Prompts through attention_varlen, their K and V into the cache, then tokens: append, attend with weights, evict."""
    lens, hq, hkv, d, budget = [40, 9, 70], 8, 2, 128, 48
    g = gen(8)
    qkv = torch.randn((sum(lens), hq + 2 * hkv, d), generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    start = starts_of(lens)
    o, lse = attn.attention_varlen(q, k, v, start)
    want = ref.varlen(q, k, v, start.tolist(), d ** -0.5, True)
    assert ((o.double() - want[0]).abs() <= want[2]).all()
    c = attn.KVCache4.empty(3, hkv, 128, d)
    c.append(k, v, seq_start=start)
    ok()
    held = list(lens)
    seen = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for step in range(12):
        new = torch.randn((3, hq + 2 * hkv, d), generator=g, device="cuda").bfloat16()
        c.append(new[:, hq:hq + hkv], new[:, hq + hkv:], first_pos=seen)
        seen += 1
        held = [n + 1 for n in held]
        assert c.length.tolist() == held
        before = c.weight.clone()
        _, _, w, *_, w_tol = ref.decode(new[:, :hq], c, held, d ** -0.5)
        o, lse = c.attend(new[:, :hq], weight_out=c.weight)
        ok()
        ro, rlse, _, tol, lse_tol, _ = ref.decode(new[:, :hq], c, held, d ** -0.5)
        assert ((o.double() - ro).abs() <= tol).all() and ((lse - rlse).abs() <= lse_tol).all()
        assert ((c.weight - before - w).abs() <= w_tol + 2e-6 * (before + w))[w > 0].all()
        check_evict(c, held, budget, 8, True)
        held = [min(n, budget) for n in held]
    # the newest tokens are still there, whatever weight they had
    for b in range(3):
        for h in range(hkv):
            assert set(range(lens[b] + 12 - 8, lens[b] + 12)) <= set(c.pos[b, h, :held[b]].tolist())


def test_graph_of_a_decode_step_and_a_side_stream():
    lens, hq, hkv, d = [60, 100], 4, 2, 64

    def step(c, q, k, v, stream=None):
        c.append(k, v, stream=stream)
        o, lse = c.attend(q, weight_out=c.weight, stream=stream)
        c.evict(90, 4, stream=stream)
        return o, lse

    x = torch.randn((2, 8, d), generator=gen(1), device="cuda").bfloat16()
    args = x[:, :4], x[:, 4:6], x[:, 6:]
    a, b, e = (filled(2, hkv, 128, d, lens, seed=9) for _ in range(3))
    want = [step(a, *args) for _ in range(4)]
    ok()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [step(b, *args, stream=side) for _ in range(4)]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(e, *args)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])
        assert torch.equal(got[i][0], want[i][0])
    for n in ("k_codes", "v_codes", "pos", "length"):
        assert torch.equal(getattr(a, n), getattr(b, n)) and torch.equal(getattr(a, n), getattr(e, n))
    assert torch.equal(a.weight.nan_to_num(-1), e.weight.nan_to_num(-1))
    ok()


@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("max_len", [2048, 2049])
@pytest.mark.parametrize("hq", [16, 18])
def test_attend_both_sides_of_the_one_launch_rule(hq, max_len, weight):
    """2048 entries a CTA a row, one more: shares; groups of 8 and 9 heads, of which the second needs two blocks."""
    lens = [2048, 1500, 0, 64, 2047]
    c = filled(5, 2, 2049, 128, lens, seed=hq)
    q = torch.randn((5, hq, 128), generator=gen(1), device="cuda").half()
    check_attend(c, q, lens, weight=weight, max_len=max_len)


@pytest.mark.parametrize("dtype,top", [(torch.bfloat16, 1e-30), (torch.bfloat16, 1e30), (torch.float16, 2.0 ** -20), (torch.float16, 65504.0)])
def test_attend_queries_of_any_size(dtype, top):
    """The largest and smallest queries: the logits' range comes back through the softmax's scale."""
    lens, D = [333, 1], 128
    c = filled(2, 2, 340, D, lens, seed=9)
    q = torch.randn((2, 8, D), generator=gen(3), device="cuda")
    q = (q / q.abs().amax() * top).to(dtype)
    check_attend(c, q, lens, scale=2.0 / top)
    c.k_meta.zero_()
    check_attend(c, q, lens, scale=1.0)
