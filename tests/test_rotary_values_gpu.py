"""qk_norm_rope, its gradient and the append to pages on values that a product with
zero would change: infinities, NaN and signed zeros in channels that are not turned.
Without a norm such a channel of the result is the input's, bit by bit."""
from __future__ import annotations

import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import rotary_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
SPECIAL = (math.inf, -math.inf, math.nan, 0.0, -0.0)


def bits(x):
    """16-bit words, every NaN as one."""
    return torch.where(x.isnan(), torch.full_like(x, math.nan), x).contiguous().view(torch.int16)


def marked(shape, dtype, rot, seed):
    """Random rows whose channels from rot on hold special values here and there."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV).to(dtype)
    at = torch.rand(shape, generator=g, device=DEV)
    at[..., :rot] = 1.0
    for i, v in enumerate(SPECIAL):
        x[(at >= 0.05 * i) & (at < 0.05 * (i + 1))] = v
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 48), (128, 0), (128, 32), (128, 96), (128, 112)])
def test_without_a_norm(d, rot, inter, dtype):
    q, k = marked((2, 33, 6, d), dtype, rot, 1), marked((2, 33, 3, d), dtype, rot, 2)
    f = attn.rotary_frequencies(rot) if rot else []
    pos = (torch.arange(33, device=DEV, dtype=torch.int32) + 700).expand(2, 33).contiguous()
    for rope in (attn.Rotary(f, interleaved=inter, amplitude=1.25),) + ((None,) if rot == 0 else ()):
        out = attn.qk_norm_rope(q, k, rope, pos)
        grads = attn.qk_norm_rope_backward(q, k, torch.ones_like(q), torch.ones_like(k), rope, pos)
        torch.cuda.synchronize()
        for x, y, dx in zip((q, k), out, grads):
            assert torch.equal(bits(y[..., rot:]), bits(x[..., rot:]))
            assert torch.equal(bits(dx[..., rot:]), bits(x[..., rot:]))
            if rot:
                part = x[..., :rot]
                want, tol = ref.forward(part, None, pos, f, inter, 1.25, 1e-6)
                assert ((y[..., :rot].double() - want).abs() <= tol).all()
                want, tol, _, _ = ref.backward(part, part, None, pos, f, inter, 1.25, 1e-6, 0)
                assert ((dx[..., :rot].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_with_a_norm(d, inter):
    """An infinity makes its own channel NaN (inf / inf) and the rest of its head zero (x / inf); NaN makes the head NaN."""
    rot = d // 2
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k = (torch.randn((1, 9, h, d), generator=g, device=DEV).half() for h in (4, 2))
    w = list((1 + 0.3 * torch.randn((2, d), generator=g, device=DEV)).half())
    pos = torch.arange(9, device=DEV, dtype=torch.int32)[None]
    rope = attn.Rotary(attn.rotary_frequencies(rot), interleaved=inter)
    want = attn.qk_norm_rope(q, k, rope, pos, *w)
    hit = [(0, 0, rot), (2, 1, d - 1), (5, 3, rot + 7)]
    for s, h, c in hit:
        q[0, s, h, c] = -math.inf if s == 2 else math.inf
    q[0, 8, 2, rot + 1] = math.nan
    got = attn.qk_norm_rope(q, k, rope, pos, *w)
    torch.cuda.synchronize()
    keep = torch.ones((9, 4), dtype=torch.bool, device=DEV)
    for s, h, c in hit:
        row = got[0][0, s, h].clone()
        assert row[c].isnan()
        row[c] = 0
        assert not row.any(), (s, h, c, row)
        keep[s, h] = False
    assert got[0][0, 8, 2].isnan().all()
    keep[8, 2] = False
    assert torch.equal(got[0][0][keep], want[0][0][keep]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 32), (128, 0), (128, 48)])
def test_append_writes_keys_as_they_are(d, rot, inter, dtype):
    """Keys (and queries) of channels that are not turned come to their pages as values do."""
    n, H, page = 40, 3, 16
    q, k, v = marked((n, 5, d), dtype, rot, 4), marked((n, H, d), dtype, rot, 5), marked((n, H, d), dtype, 0, 6)
    cache = attn.PagedKVCache.empty(1, H, 4, page, 4, d, dtype)
    cache.page_table.copy_(torch.tensor([[2, 0, 3, 1]], dtype=torch.int32))
    rope = attn.Rotary(attn.rotary_frequencies(rot), interleaved=inter) if rot else None
    q_out = cache.append(k, v, seq_start=torch.tensor([0, n], dtype=torch.int32, device=DEV), q=q, rope=rope)
    torch.cuda.synchronize()
    j = torch.arange(n, device=DEV)
    where = cache.page_table[0].long()[j // page]
    kk, vv = cache.k_pages[where, :, j % page], cache.v_pages[where, :, j % page]
    assert torch.equal(bits(q_out[..., rot:]), bits(q[..., rot:]))
    assert torch.equal(bits(kk[..., rot:]), bits(k[..., rot:])) and torch.equal(bits(vv), bits(v))


def test_outputs_whose_rows_overlap_are_refused():
    q, k = (torch.randn((2, 5, 4, 64), device=DEV).bfloat16() for _ in range(2))
    buffer = torch.zeros(4000, dtype=torch.bfloat16, device=DEV)
    for strides in ((5 * 4 * 64, 4 * 64, 32, 1), (640, 64, 64, 1), (1024, 256, 64, 1)):
        bad = buffer.as_strided(q.shape, strides)
        for name in ("q_out", "k_out"):
            with pytest.raises(ValueError, match="apart"):
                attn.qk_norm_rope(q, k, None, **{name: bad})
        for name in ("dq", "dk"):
            with pytest.raises(ValueError, match="apart"):
                attn.qk_norm_rope_backward(q, k, q, k, None, **{name: bad})
    assert not buffer.any()
