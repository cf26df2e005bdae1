"""Inputs at the edges of what the serving calls take, each against its 64-bit
definition."""
from __future__ import annotations

import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ok():
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK


def starts_of(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


# --- packed prompts --------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nats,at", [(6, 0), (12, 0), (16, 0), (18, 0), (18, 500), (20, 700)])
def test_fp16_prompt_of_keys_far_below_the_maximum(nats, at, D, causal):
    """One key takes nearly all the weight and has V = 0, so O is what thousands of keys e^-nats as heavy add up to.

    The bound.  p is held as 2^11 p relative to the row's reference, whose own key has p = 1, so l >= 1; fp16 is exact
    to 2^-25 where it is subnormal: an absolute 2^-36 a key and |v|, on top of the relative half step of ref.varlen.
    """
    n, scale = 4096, 0.125
    q = torch.zeros((n, 2, D), device="cuda")
    q[..., 0] = 8.0
    k = torch.zeros((n, 1, D), device="cuda")
    k[at, :, 0] = nats
    v = 1000 * (1 + torch.rand((n, 1, D), generator=gen(1), device="cuda"))
    v[at] = 0
    q, k, v = q.half(), k.half(), v.half()
    o, lse = attn.attention_varlen(q, k, v, starts_of([n]), scale=scale, causal=causal)
    ok()
    ro, rlse, tol, lse_tol = ref.varlen(q, k, v, [0, n], scale, causal)
    size = v.double().abs().cumsum(0) if causal else v.double().abs().sum(0, keepdim=True)
    assert ((lse.double() - rlse).abs() <= lse_tol).all()
    bad = (o.double() - ro).abs() > tol + 2.0 ** -36 * size
    assert not bad.any(), (int(bad.sum()), ((o.double() - ro).abs() / ro.abs().clamp(min=1e-30)).max())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_fp16_prompt_of_the_largest_values(D, causal):
    """O is a mean of V: where every V is fp16's largest number it is that number, whatever the rounding of P.

    All keys but the first have p = (1 + 1.02 * 2^-11) / 2, just above the middle of two fp16 numbers: rounded, their
    sum exceeds the row's by nearly 2^-11, and 65504 * (1 + 2^-11) would round to infinity.
    """
    n = 400
    q = torch.zeros((n, 4, D), device="cuda")
    q[..., 0] = 8.0
    k = torch.zeros((n, 2, D), device="cuda")
    k[0, :, 0] = 8.0
    v = torch.full((n, 2, D), 65504.0, device="cuda")
    v[:, 1] = -65504.0
    scale = (1 - math.log2(1 + 1.02 * 2.0 ** -11)) * math.log(2) / 64
    o, _ = attn.attention_varlen(q.half(), k.half(), v.half(), starts_of([n]), scale=scale, causal=causal)
    ok()
    want = v.repeat_interleave(2, 1).double()
    assert ((o.double() - want).abs() <= 2 * 2.0 ** -11 * 65504).all()  # P's half step and the result's


@pytest.mark.parametrize("H", [1, 200])
@pytest.mark.parametrize("starts", [[-(1 << 31), 20, (1 << 31) - 1], [0, 50, -(1 << 31), 64], [(1 << 31) - 1, -(1 << 31)],
                                    [5, -(1 << 31), -1, 40, 64], [-(1 << 31), (1 << 31) - 1]], ids=str)
def test_prompt_starts_of_any_value(starts, H):
    """With one key head each CTA finds its unit itself, with 200 the units are listed: in both, starts count as the
    rows there are (0 .. 64), and a sequence that then ends before it begins is empty."""
    total = 64
    x = torch.randn((total, 3 * H, 64), generator=gen(3), device="cuda").bfloat16()
    q, k, v = x[:, :H], x[:, H:2 * H], x[:, 2 * H:]
    out = torch.full((total, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, total), 7.0, device="cuda")
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    assert (attn.attn_fwd_varlen_workspace_bytes(total, len(starts) - 1, H, H, 64) > 16) == (H == 200)
    attn.attention_varlen(q, k, v, s, out=out, lse=lse)
    ok()
    want = [min(max(a, 0), total) for a in starts]
    heads = list(range(H)) if H == 1 else [0, 99, 199]
    pick = torch.tensor(heads, device="cuda")
    seen = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, b in zip(want, want[1:]):
        if a >= b:
            continue
        # (sequences that overlap are computed each for itself: only rows of one are looked at)
        alone = [r for r in range(a, b) if sum(c <= r < d for c, d in zip(want, want[1:])) == 1]
        ro, rlse, tol, lse_tol = ref.varlen(q[:, pick], k[:, pick], v[:, pick], [a, b], 0.125, True)
        assert ((out[alone][:, pick].double() - ro[alone]).abs() <= tol[alone]).all()
        assert ((lse[pick][:, alone].double() - rlse[:, alone]).abs() <= lse_tol[:, alone]).all()
        seen[a:b] = True
    assert (out[~seen] == 7.0).all() and (lse[:, ~seen] == 7.0).all()


# --- the cache -------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("B,H,cap", [(1, 1, 1), (1, 1, 5), (3, 1, 7), (1, 3, 129)])
def test_caches_of_an_odd_number_of_entries(B, H, cap):
    D = 64
    c = attn.KVCache4.empty(B, H, cap, D)
    x = torch.randn((B, H, D), generator=gen(1), device="cuda").bfloat16()
    c.append(x, x)
    o, lse = c.attend(x, weight_out=c.weight)
    k, v = c.read(dtype=torch.float32)
    c.evict(1)
    ok()
    code, s, m = ref.quantise(x)
    want = ref.values(ref.pack(code), torch.stack([s, m], -1))
    assert torch.equal(k.double(), want) and torch.equal(v.double(), want)
    assert ((o.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * want.abs().amax() * 4).all()
    assert c.length.tolist() == [1] * B and ((c.weight[..., 0] - 1).abs() <= 1e-6).all()


def test_buffers_can_be_exchanged_and_sizes_cannot():
    B, H, cap, D = 2, 1, 20, 64
    c = attn.KVCache4.empty(B, H, cap, D)
    old = {name: getattr(c, name) for name in ("k_codes", "k_meta", "v_codes", "v_meta", "weight", "pos", "length")}
    for name in ("k_codes", "k_meta", "v_codes", "v_meta"):
        old[name].zero_()
    x = torch.randn((B, H, D), generator=gen(1), device="cuda").bfloat16()
    c.append(x, x)
    # what a call has written elsewhere takes the old buffer's place
    grown = torch.empty_like(c.length)
    c.append(x, x, length_out=grown)
    c.length = grown
    weight = torch.full_like(c.weight, 3.0)
    c.attend(x, weight_out=weight)
    c.weight = weight
    c.append(x, x)
    ok()
    assert c.length is grown and grown.tolist() == [3, 3] and old["length"].tolist() == [1, 1]
    assert (old["weight"] == 0).all() and (weight[:, :, 2] == 0).all() and ((weight[:, :, :2] - 0.5).abs() <= 1e-6).all()
    for slot, name in enumerate(("k_codes", "k_meta", "v_codes", "v_meta", "pos"), 4):
        setattr(c, name, old[name].clone())
        before = old[name].clone()
        c.length.fill_(slot)  # a slot that no append before has written
        c.append(-x, -x)
        ok()
        assert torch.equal(old[name], before) and not torch.equal(getattr(c, name)[:, :, slot], before[:, :, slot]), name
    for name, bad in (("length", torch.zeros(3, dtype=torch.int32, device="cuda")), ("weight", weight.double()), ("pos", None),
                      ("weight", weight[..., ::2]), ("k_codes", old["k_codes"].cpu())):
        with pytest.raises((ValueError, TypeError)):
            setattr(c, name, bad)
    for name in ("B", "H_kv", "capacity", "D", "device"):
        with pytest.raises(AttributeError):
            setattr(c, name, 1)
    with pytest.raises(AttributeError):
        del c.weight
    assert c.weight is weight and c.length is grown


def test_a_copied_cache_has_buffers_of_its_own_only_where_it_is_deep():
    import copy

    c = attn.KVCache4.empty(1, 1, 4, 64)
    x = torch.randn((1, 1, 64), generator=gen(1), device="cuda").bfloat16()
    c.append(x, x)
    shallow, deep = copy.copy(c), copy.deepcopy(c)
    shallow.length = torch.zeros_like(c.length)  # the copy's alone
    c.append(x, x)
    deep.append(-x, -x)
    ok()
    assert shallow.k_codes is c.k_codes and shallow.length.tolist() == [0]
    assert c.length.tolist() == [2] and deep.length.tolist() == [2]
    assert torch.equal(deep.k_codes[:, :, 0], c.k_codes[:, :, 0]) and not torch.equal(deep.k_meta[:, :, 1], c.k_meta[:, :, 1])


@pytest.mark.parametrize("low,high", [(-3e38, 3e38), (-3.38e38, 1e38), (0.0, 3.38e38), (-3.38e38, -1e38), (-1e31, 2e31)])
@pytest.mark.parametrize("D", [64, 128])
def test_append_of_the_largest_finite_values(D, low, high):
    """A group is finite where its values are, also where max - min is beyond fp32's range."""
    n, H = 64, 2
    x = (low + (high / 2 - low / 2) * 2 * torch.rand((n, H, D), generator=gen(1), device="cuda", dtype=torch.float64)).bfloat16()
    x[:, :, 3::64], x[:, :, 40::64] = low, high
    c = attn.KVCache4.empty(1, H, n, D)
    c.append(x, x.flip(0), seq_start=starts_of([n]))
    ok()
    for y, codes, meta in ((x, c.k_codes, c.k_meta), (x.flip(0), c.v_codes, c.v_meta)):
        code, s, m = ref.quantise(y.transpose(0, 1))
        assert s.isfinite().all() and torch.equal(meta[0].double(), torch.stack([s, m], -1))
        q = ((y.transpose(0, 1).double().unflatten(-1, (-1, 64)) - m[..., None]) / s[..., None]).flatten(-2)
        near = (q - q.floor() - 0.5).abs() <= 16 * 2.0 ** -23  # a 32-bit quotient may fall on the half way point itself
        got = ref.unpack(codes[0])
        assert torch.equal(got[~near], code[~near]) and ((got - code).abs()[near] <= 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_and_read_of_the_smallest_scales(dtype):
    """Scales below 2^-100, subnormal ones among them, and 0: the read's own branch, and the append's division."""
    n, D = 48, 128
    x = torch.randn((n, 1, D), generator=gen(4), device="cuda", dtype=torch.float64)
    x *= (2.0 ** torch.linspace(-131, -96, n, device="cuda", dtype=torch.float64))[:, None, None]
    x[0] = 0
    x = x.bfloat16()
    c = attn.KVCache4.empty(1, 1, n, D)
    c.append(x, x, seq_start=starts_of([n]))
    k, _ = c.read(seq_start=starts_of([n]), rows=n, dtype=dtype)
    ok()
    code, s, m = ref.quantise(x.transpose(0, 1))
    assert (s < 2.0 ** -100).any() and ((s > 0) & (s < 2.0 ** -126)).any() and (s > 2.0 ** -100).any() and (s == 0).any()
    assert torch.equal(c.k_meta[0].double(), torch.stack([s, m], -1))
    want = ref.values(c.k_codes, c.k_meta)[0].transpose(0, 1)
    # one rounding to fp32, and one to the output's type; subnormal steps below the normal numbers
    u = ref.HALF_STEP[torch.float32] + (ref.HALF_STEP[dtype] if dtype != torch.float32 else 0)
    assert ((k.double() - want).abs() <= u * want.abs() + (2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -150)).all()
    q = ((x.transpose(0, 1).double().unflatten(-1, (-1, 64)) - m[..., None]) / s[..., None].where(s[..., None] != 0, torch.ones_like(s[..., None]))).flatten(-2)
    near = (q - q.floor() - 0.5).abs() <= 2.0 ** -19
    assert torch.equal(ref.unpack(c.k_codes[0])[~near], code[~near])


def test_a_drop_outlives_the_report_of_another_failure():
    c = attn.KVCache4.empty(1, 1, 1, 128)
    x = torch.zeros((2, 1, 128), dtype=torch.bfloat16, device="cuda")
    ok()
    c.append(x, x, seq_start=starts_of([2]))
    torch.cuda.synchronize()
    # the self-test waits its limit out and returns: its report comes first, the drop's stays for the next call
    assert attn.attn_watchdog_selftest(1_000_000) == attn.ATTN_ERR_TIMEOUT
    assert attn.attn_fwd_debug_status() == attn.ATTN_ERR_CAPACITY
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("n", [200, 1900, 9000])
def test_attend_values_of_very_unlike_scales(n, order, D, dtype):
    """Keys of little weight have the largest scales in V: what the heavy keys add has to keep its bits.

    Half of the keys' scales are 2^e, e up to 48, at a weight of 4^-e; a second head gives the largest scales the largest
    weights, 2^e.  The bound: p s is held in fp16 to 2^-36 of at most twice the largest p s of its head (subnormals),
    times |c - 8| <= 8, on top of ref.decode's relative half step.
    """
    g = gen(n)
    e = torch.randint(0, 49, (n,), generator=g, device="cuda").float()
    e[torch.rand(n, generator=g, device="cuda") < 0.5] = 0
    e[:3] = torch.tensor([48.0, 0.0, 24.0])
    if order != "mixed":
        e = e.sort(descending=order == "falling")[0]
    c = attn.KVCache4.empty(1, 1, n, D)
    code, s, m = ref.quantise(torch.randn((1, 1, n, D), generator=g, device="cuda").bfloat16())
    c.v_codes.copy_(ref.pack(code))
    c.v_meta.copy_(torch.stack([s, m], -1) * (2.0 ** e)[:, None, None])
    c.k_codes.zero_()
    c.k_meta.zero_()
    c.k_meta[..., 1] = -e[:, None]  # every channel of key j is -e_j
    c.length.fill_(n)
    q = torch.zeros((1, 2, D), device="cuda")
    q[0, 0, 0], q[0, 1, 0] = 2.0, -1.0
    q = q.to(dtype)
    o, lse = c.attend(q, scale=math.log(2))
    ok()
    ro, rlse, _, tol, lse_tol, _ = ref.decode(q, c, [n], math.log(2))
    x = -e.double()[None] * torch.tensor([[2.0], [-1.0]], device="cuda", dtype=torch.float64) * math.log(2)
    ps = (torch.softmax(x, 1)[..., None] * c.v_meta[0, 0, :, :, 0].double()[None]).amax(1)  # [head, group]
    tol = tol + (n * 8 * 2.0 ** -35 * ps).repeat_interleave(64, 1)
    keep = ro.abs() < 60000 if dtype == torch.float16 else torch.ones_like(ro, dtype=torch.bool)
    bad = ((o.double() - ro).abs() > tol) & keep
    assert not bad.any(), (int(bad.sum()), ((o.double() - ro).abs() / tol)[keep].max())
    assert ((lse.double() - rlse).abs() <= lse_tol).all()


def filled(B, H, cap, D, n, seed):
    """A cache whose first n entries of every row are random."""
    c = attn.KVCache4.empty(B, H, cap, D)
    x = torch.randn((2, B, H, n, D), generator=gen(seed), device="cuda")
    for codes, meta, y in ((c.k_codes, c.k_meta, x[0]), (c.v_codes, c.v_meta, x[1])):
        code, s, m = ref.quantise(y.bfloat16())
        codes[:, :, :n] = ref.pack(code)
        meta[:, :, :n] = torch.stack([s, m], -1).bfloat16()
    c.weight[:, :, :n] = torch.rand((B, H, n), generator=gen(seed + 1), device="cuda")
    c.pos[:, :, :n] = torch.arange(n, dtype=torch.int32, device="cuda")
    c.length.fill_(n)
    return c


def test_two_threads_on_one_stream():
    """Calls of two threads, each on a cache of its own, whose launches may interleave on the stream they share."""
    import threading

    B, H, cap, D = 3, 2, 6000, 128
    caches = [filled(B, H, cap, D, 5000, seed) for seed in (1, 2)]
    q = torch.randn((B, 8, D), generator=gen(3), device="cuda").bfloat16()
    caches[1].length.copy_(torch.tensor([5, 0, 4999], dtype=torch.int32))
    want = [c.attend(q, weight_out=torch.zeros_like(c.weight)) for c in caches]
    ok()
    got = [[], []]

    def work(i):
        for _ in range(40):
            got[i].append(caches[i].attend(q, weight_out=torch.zeros_like(caches[i].weight)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    for i in range(2):
        assert len(got[i]) == 40
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


# --- offsets beyond 32 bits ------------------------------------------------------------------------------------------

def test_cache_offsets_beyond_32_bits():
    """More than 2^33 bytes of codes a buffer, so that the last sequence's lie beyond 2^31 four-byte words, too: append,
    read, attention in one launch and in shares, with and without weights, and eviction, all on that sequence."""
    B, H, cap, D, n = 18, 8, 1 << 20, 128, 5000
    small = filled(1, H, n, D, n, seed=5)
    c = attn.KVCache4.empty(B, H, cap, D)
    last = B - 1
    assert c.k_codes.stride(0) * last // 4 > 1 << 31 and c.k_codes.stride(0) * last > 1 << 32
    names = ("k_codes", "k_meta", "v_codes", "v_meta", "weight", "pos")
    lens = [3] + [0] * (B - 2) + [n]
    for name in names:
        getattr(c, name)[last, :, :n] = getattr(small, name)[0]
        getattr(c, name)[0, :, :3] = getattr(small, name)[0, :, :3]
    c.length.copy_(torch.tensor(lens, dtype=torch.int32))
    q = torch.randn((B, 16, D), generator=gen(1), device="cuda").bfloat16()
    for held, max_len in ((n, None), (n, n), (200, 200)):  # the capacity's shares, the length's, one launch
        if held < n:
            small.length.fill_(held)
        ro, rlse, rw, tol, lse_tol, w_tol = ref.decode(q[last:], small, [held], D ** -0.5)
        for weight in (False, True):
            out = torch.zeros_like(c.weight) if weight else None
            o, lse = c.attend(q, weight_out=out, max_len=max_len)
            ok()
            assert ((o[last].double() - ro[0]).abs() <= tol[0]).all() and ((lse[last].double() - rlse[0]).abs() <= lse_tol[0]).all()
            assert (o[1:last] == 0).all() and (lse[1:last] == -math.inf).all()
            if weight:
                err = (out[last, :, :held].double() - small.weight[0, :, :held].double() - rw[0, :, :held]).abs()
                assert (err <= w_tol[0, :, :held] + 2.0 ** -23 * (small.weight[0, :, :held].double() + rw[0, :, :held])).all()
                assert (out[last, :, held:] == 0).all()
                del out
    x = torch.randn((B, H, D), generator=gen(2), device="cuda").bfloat16()
    c.append(x, x)
    k, v = c.read(first_slot=torch.tensor(lens, dtype=torch.int32, device="cuda"), dtype=torch.float32)
    ok()
    code, s, m = ref.quantise(x)
    want = ref.values(ref.pack(code), torch.stack([s, m], -1))
    assert torch.equal(k.double(), want) and torch.equal(v.double(), want)
    assert c.length.tolist() == [a + 1 for a in lens] and (c.pos[last, :, n] == n).all()
    before = {name: getattr(c, name)[last, :, :n + 1].clone() for name in names}
    budget, recent = 3000, 50
    c.evict(budget, recent, max_len=n + 1)
    ok()
    assert c.length.tolist() == [min(a + 1, budget) for a in lens]
    for h in range(H):
        src = torch.tensor(ref.evict(before["weight"][h].tolist(), before["pos"][h].tolist(), n + 1, budget, recent), device="cuda")
        for name in names:
            assert torch.equal(getattr(c, name)[last, h, :budget], before[name][h, src]), name


def test_prompt_offsets_beyond_32_bits():
    """Rows that lie beyond 2^32 bytes and 2^31 elements of q, k, v and o."""
    total, hq, hkv, d, lens = 1_200_000, 16, 1, 128, [37, 300]
    first = total - sum(lens)
    x = torch.empty((total, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    x[first:] = torch.randn((sum(lens), hq + 2 * hkv, d), generator=gen(6), device="cuda").bfloat16()
    out = torch.zeros((total, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((hq, total), device="cuda")
    assert first * hq * d > 1 << 31 and first * hq * d * 2 > 1 << 32
    starts = torch.tensor([first, first + lens[0], total], dtype=torch.int32, device="cuda")
    attn.attention_varlen(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], starts, out=out, lse=lse)
    ok()
    y = x[first:]
    ro, rlse, tol, lse_tol = ref.varlen(y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], [0, lens[0], sum(lens)], d ** -0.5, True)
    assert ((out[first:].double() - ro).abs() <= tol).all() and ((lse[:, first:].double() - rlse).abs() <= lse_tol).all()
    assert not out[:first].any() and not lse[:, :first].any()


@pytest.mark.parametrize("ratio", [1, 16, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_logits_are_as_exact_as_fp32_products(D, dtype, ratio):
    """A sequence of one entry has its logit as LSE.  Its rounding errors, relative to sum |q||k|, are those of fp32 sums:
    over 4096 rows their root mean square is at most three times a plain fp32 product's (two, should an adder truncate,
    and three operations more), also where one channel of q is `ratio` times the others."""
    B, G = 512, 8
    c = filled(B, 1, 1, D, 1, seed=11)
    q = torch.randn((B, G, D), generator=gen(12), device="cuda")
    q[..., 5] *= ratio
    q = q.to(dtype)
    _, lse = c.attend(q, scale=1.0)
    ok()
    k = ref.values(c.k_codes, c.k_meta)[:, 0, 0]
    want, reach = (q.double() * k[:, None]).sum(-1), (q.double().abs() * k[:, None].abs()).sum(-1)
    plain = (q.float() @ k.float()[:, :, None])[..., 0]
    off = [((x.double() - want) / reach).square().mean().sqrt() for x in (lse, plain)]
    assert off[0] <= 3 * off[1], off


@pytest.mark.parametrize("power", [-100, -40, 40, 100])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1000, 5000])
def test_attend_values_times_a_power_of_two(n, D, power):
    """Every step is exact in powers of two, so V times 2^power gives O times 2^power, bit by bit."""
    c = filled(2, 2, n, D, n, seed=13)
    q = 3 * torch.randn((2, 6, D), generator=gen(14), device="cuda").bfloat16()
    o, lse = c.attend(q)
    c.v_meta = c.v_meta * 2.0 ** power
    o2, lse2 = c.attend(q)
    ok()
    assert torch.equal(lse, lse2) and torch.equal(o.double() * 2.0 ** power, o2.double())


def test_attend_nan_values_stay_in_their_channels():
    """An entry whose V is not finite in one group of channels: those channels alone; in K: the heads that see it."""
    for n in (100, 5000):
        c = filled(2, 2, n, 128, n, seed=15)
        q = torch.randn((2, 8, 128), generator=gen(16), device="cuda").bfloat16()
        good, lse = c.attend(q)
        c.v_meta[1, 0, n // 2, 1] = math.nan
        o, z = c.attend(q)
        ok()
        assert o[1, :4, 64:].isnan().all() and torch.equal(z, lse)
        assert torch.equal(o[1, :4, :64], good[1, :4, :64]) and torch.equal(o[1, 4:], good[1, 4:]) and torch.equal(o[0], good[0])
        c.v_meta[1, 0, n // 2, 1] = 1.0
        c.k_meta[0, 1, 3, 0] = math.nan
        o, z = c.attend(q)
        ok()
        assert o[0, 4:].isnan().all() and z[0, 4:].isnan().all() and torch.equal(o[0, :4], good[0, :4]) and torch.equal(z[1], lse[1])
