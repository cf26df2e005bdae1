"""qk_norm_rope and its gradient against the 64-bit definition: layouts, parts of
heads, types, strides, positions, sizes from one row to many; streams, graphs, and
the call before and behind attention."""
from __future__ import annotations

import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import rotary_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make(B, S, hq, hk, d, dtype, seed=0, far=0, weights="same"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn((B, S, hq + 2 * hk, d), generator=g, device=DEV).to(dtype)
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    w_type = dtype if weights == "same" else torch.float32
    w = [None, None] if weights is None else list((1 + 0.3 * torch.randn((2, d), generator=g, device=DEV)).to(w_type))
    pos = (torch.randint(0, far + 1, (B, 1), generator=g, device=DEV) + torch.arange(S, device=DEV)).int()
    dq, dk = (torch.randn((B, h, S, d), generator=g, device=DEV).to(dtype).transpose(1, 2) for h in (hq, hk))
    return q, k, pos, w, dq, dk


def chain(B, S, hq, hk, d):
    """Rows that a lane adds up at most: a block's share of the tokens, eight warps taking a token's groups of heads in turn."""
    rows = 32 // (d // 8)
    groups = -(-hq // rows) + -(-hk // rows)
    tiles = B * -(-S // 8)
    return -(-tiles // 608) * (-(-8 * groups // 8) + 1) + groups


def check(got, want, tol, what):
    assert got.isfinite().all(), what
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), ((got.double() - want).abs() / tol).max())


def both(B, S, hq, hk, d, dtype, rot, inter, weights="same", amp=1.0, far=0, seed=0, eps=1e-6, freqs=None):
    q, k, pos, w, dq, dk = make(B, S, hq, hk, d, dtype, seed, far, weights)
    freqs = (attn.rotary_frequencies(rot) if rot else []) if freqs is None else freqs
    rope = attn.Rotary(freqs, interleaved=inter, amplitude=amp) if freqs else None
    out = attn.qk_norm_rope(q, k, rope, pos, q_weight=w[0], k_weight=w[1], eps=eps)
    grads = attn.qk_norm_rope_backward(dq, dk, q, k, rope, pos, q_weight=w[0], k_weight=w[1], eps=eps)
    torch.cuda.synchronize()
    n = chain(B, S, hq, hk, d)
    for i, (x, dy, name) in enumerate(((q, dq, "q"), (k, dk, "k"))):
        y, tol = ref.forward(x, w[i], pos, freqs, inter, amp, eps)
        check(out[i], y, tol, name)
        dx, tol, dw, dw_tol = ref.backward(dy, x, w[i], pos, freqs, inter, amp, eps, n)
        check(grads[i], dx, tol, "d" + name)
        if dw is None:
            assert grads[2 + i] is None
        else:
            check(grads[2 + i], dw, dw_tol, "dw of " + name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (64, 0), (128, 128), (128, 16), (128, 32), (128, 96), (128, 112)])
def test_layouts_and_parts(d, rot, inter, dtype):
    both(2, 19, 6, 3, d, dtype, rot, inter, amp=1.25, far=5000, seed=rot)


@pytest.mark.parametrize("weights", [None, "same", "float32"])
@pytest.mark.parametrize("B,S,hq,hk", [(1, 1, 1, 1), (1, 2, 3, 1), (5, 1, 32, 8), (1, 7, 128, 8), (3, 9, 5, 5), (1, 333, 14, 2), (64, 3, 8, 1),
                                       (2, 1111, 32, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_sizes(d, B, S, hq, hk, weights):
    both(B, S, hq, hk, d, torch.bfloat16, d, False, weights, seed=S)


def test_one_of_the_weights():
    q, k, pos, w, dq, dk = make(1, 40, 4, 2, 64, torch.bfloat16)
    f = attn.rotary_frequencies(64)
    rope = attn.Rotary(f)
    for i in range(2):
        ww = [w[0], None] if i == 0 else [None, w[1]]
        out = attn.qk_norm_rope(q, k, rope, pos, *ww)
        grads = attn.qk_norm_rope_backward(dq, dk, q, k, rope, pos, *ww)
        assert grads[3 - i] is None and grads[2 + i] is not None
        for j, (x, dy) in enumerate(((q, dq), (k, dk))):
            check(out[j], *ref.forward(x, ww[j], pos, f, False, 1.0, 1e-6), "out")
            dx, tol, dw, dw_tol = ref.backward(dy, x, ww[j], pos, f, False, 1.0, 1e-6, chain(1, 40, 4, 2, 64))
            check(grads[j], dx, tol, "dx")
            if dw is not None:
                check(grads[2 + j], dw, dw_tol, "dw")


def test_far_positions():
    """Angles of 10^9 radians; negative positions; frequencies above a turn and below zero."""
    f = [1.0, 7.5, -0.3, 0.01, 1e-4, 2.0, 1e-8, 0.5]
    q, k, _, w, _, _ = make(1, 6, 2, 1, 64, torch.float16, seed=3)
    pos = torch.tensor([[0, 1 << 30, (1 << 31) - 1, -1, -(1 << 31), 123456789]], dtype=torch.int32, device=DEV)
    out = attn.qk_norm_rope(q, k, attn.Rotary(f), pos, w[0], w[1])
    # in 64 bits the reference's own angles are off by 2^-53 of 1.6e10
    for i, x in enumerate((q, k)):
        y, tol = ref.forward(x, w[i], pos, f, False, 1.0, 1e-6)
        check(out[i], y, tol + 4e-6 * ref.reach(y, f, False, 1.0), "far")


def test_no_rows():
    q, k = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV), torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    pos, w = torch.empty(0, dtype=torch.int32, device=DEV), torch.ones(64, dtype=torch.bfloat16, device=DEV)
    rope = attn.Rotary(attn.rotary_frequencies(64))
    a, b = attn.qk_norm_rope(q, k, rope, pos, w, w)
    assert a.shape == q.shape and b.shape == k.shape
    dq, dk, dqw, dkw = attn.qk_norm_rope_backward(q, k, q, k, rope, pos, w, w)
    torch.cuda.synchronize()
    assert dq.shape == q.shape and not dqw.any() and not dkw.any()


@pytest.mark.parametrize("inter", [False, True])
def test_outputs_of_any_strides_and_in_place(inter):
    q, k, pos, w, dq, dk = make(2, 70, 8, 4, 64, torch.bfloat16, seed=8)
    rope = attn.Rotary(attn.rotary_frequencies(32), interleaved=inter)
    want = attn.qk_norm_rope(q, k, rope, pos, *w)
    grads = attn.qk_norm_rope_backward(dq, dk, q, k, rope, pos, *w)
    # [B, H, S, D], and heads that lie apart
    q_out = torch.empty((2, 8, 70, 64), dtype=q.dtype, device=DEV).transpose(1, 2)
    wide = torch.full((2, 70, 4, 128), 5.0, dtype=k.dtype, device=DEV)
    a, b = attn.qk_norm_rope(q, k, rope, pos, *w, q_out=q_out, k_out=wide[..., :64])
    assert a is q_out and torch.equal(a, want[0]) and torch.equal(b, want[1]) and (wide[..., 64:] == 5.0).all()
    ga, gb = dq.clone(), dk.clone()
    got = attn.qk_norm_rope_backward(ga, gb, q, k, rope, pos, *w, dq=ga, dk=gb)
    for x, y in zip(got, grads):
        assert torch.equal(x, y)
    qq, kk = q, k  # slices of one buffer, written where they are
    attn.qk_norm_rope(qq, kk, rope, pos, *w, q_out=qq, k_out=kk)
    assert torch.equal(qq, want[0]) and torch.equal(kk, want[1])
    # three dimensions are one batch
    x, y = attn.qk_norm_rope(want[0][1], want[1][1], rope, pos[1], *w)
    z, _ = attn.qk_norm_rope(want[0][1:], want[1][1:], rope, pos[1:], *w)
    assert torch.equal(x, z[0])


def test_extreme_rows():
    """Rows of zeros, of the type's largest numbers and of NaN: their own results alone tell."""
    q, k, pos, w, dq, dk = make(1, 12, 4, 2, 64, torch.bfloat16, seed=4)
    q, k = q.contiguous(), k.contiguous()
    f = attn.rotary_frequencies(64)
    rope = attn.Rotary(f)
    want = attn.qk_norm_rope(q, k, rope, pos, *w)
    q[0, 3] = 0
    q[0, 5, 1] = math.nan
    k[0, 7, 0, 9] = math.inf
    got = attn.qk_norm_rope(q, k, rope, pos, *w)
    assert not got[0][0, 3].any()
    assert got[0][0, 5, 1].isnan().all() and not got[1][0, 7, 0].isfinite().all()
    keep_q, keep_k = torch.ones((12, 4), dtype=torch.bool, device=DEV), torch.ones((12, 2), dtype=torch.bool, device=DEV)
    keep_q[3], keep_q[5, 1], keep_k[7, 0] = False, False, False
    assert torch.equal(got[0][0][keep_q], want[0][0][keep_q]) and torch.equal(got[1][0][keep_k], want[1][0][keep_k])


def test_the_same_from_call_to_call_streams_and_graph():
    q, k, pos, w, dq, dk = make(1, 3000, 16, 4, 64, torch.bfloat16, seed=6)
    rope = attn.Rotary(attn.rotary_frequencies(64))
    want = (*attn.qk_norm_rope(q, k, rope, pos, *w), *attn.qk_norm_rope_backward(dq, dk, q, k, rope, pos, *w))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = (*attn.qk_norm_rope(q, k, rope, pos, *w, stream=side),
           *attn.qk_norm_rope_backward(dq, dk, q, k, rope, pos, *w, stream=side))
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = (*attn.qk_norm_rope(q, k, rope, pos, *w), *attn.qk_norm_rope_backward(dq, dk, q, k, rope, pos, *w))
    for _ in range(2):
        for x in held:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y)


def test_python_refusals_on_the_device():
    q, k, pos, w, dq, dk = make(1, 8, 4, 2, 64, torch.bfloat16)
    rope = attn.Rotary(attn.rotary_frequencies(64))
    for bad in (dict(positions=None), dict(positions=pos.long()), dict(positions=pos[:, :7]), dict(q_weight=w[0][:32]),
                dict(q_weight=w[0].double()), dict(q_out=torch.empty_like(q)[:, :7]), dict(k_out=k.float()),
                dict(q_out=torch.empty((1, 8, 1, 64), dtype=q.dtype, device=DEV).expand(1, 8, 4, 64))):
        with pytest.raises(ValueError):
            attn.qk_norm_rope(q, k, rope, **{**dict(positions=pos, q_weight=w[0], k_weight=w[1]), **bad})
    with pytest.raises(TypeError):
        attn.qk_norm_rope(q, k, rope, pos, w[0].float(), w[1])
    with pytest.raises(attn.AttnError):
        attn.qk_norm_rope(q, k, rope, pos, *w, eps=-1.0)
    with pytest.raises(ValueError, match="rotation"):
        attn.qk_norm_rope(q, k, attn.Rotary([1.0] * 8, device="cpu"), pos)
    with pytest.raises(attn.AttnError):  # rows that do not begin on 16 bytes
        x = torch.empty(8 * 4 * 64 + 1, dtype=q.dtype, device=DEV)[1:].view(8, 4, 64)
        attn.qk_norm_rope(x, x, rope, pos[0])


def test_training_step_through_attention():
    """Projection's rows -> norm and rotation -> dense causal attention -> its gradients -> gradients of the rows and the weights."""
    B, S, H, D = 2, 384, 4, 64
    g = torch.Generator(device=DEV).manual_seed(12)
    qkv = torch.randn((B, S, 3, H, D), generator=g, device=DEV).bfloat16()
    w = list((1 + 0.2 * torch.randn((2, D), generator=g, device=DEV)).bfloat16())
    d_o = torch.randn((B, H, S, D), generator=g, device=DEV).bfloat16()
    pos = torch.arange(S, device=DEV, dtype=torch.int32).expand(B, S).contiguous()
    f = attn.rotary_frequencies(D)
    rope = attn.Rotary(f)
    dense = [torch.empty((B, H, S, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    attn.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], rope, pos, *w, q_out=dense[0].transpose(1, 2), k_out=dense[1].transpose(1, 2))
    v = qkv[:, :, 2].transpose(1, 2).contiguous()
    o, lse = attn.attention_forward(*dense, v, causal=True)
    dq, dk, dv = attn.attention_backward(*dense, v, o, lse, d_o, causal=True)
    grad = torch.empty_like(qkv)
    _, _, dqw, dkw = attn.qk_norm_rope_backward(dq.transpose(1, 2), dk.transpose(1, 2), qkv[:, :, 0], qkv[:, :, 1], rope, pos, *w,
                                                dq=grad[:, :, 0], dk=grad[:, :, 1])
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    # the same in 64 bits, by autograd
    leaves = [qkv[:, :, 0].double().requires_grad_(), qkv[:, :, 1].double().requires_grad_(), w[0].double().requires_grad_(),
              w[1].double().requires_grad_()]
    turned = []
    for x, ww in ((leaves[0], leaves[2]), (leaves[1], leaves[3])):
        z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * ww
        t = pos.double()[..., None, None] * torch.tensor(f, dtype=torch.float64, device=DEV)
        a, b = z[..., :D // 2], z[..., D // 2:]
        turned.append(torch.cat([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1).transpose(1, 2))
    s = turned[0] @ turned[1].transpose(-1, -2) / math.sqrt(D)
    s = s.masked_fill(torch.ones((S, S), dtype=torch.bool, device=DEV).triu(1), -math.inf)
    (torch.softmax(s, -1) @ v.double() * d_o.double()).sum().backward()
    # the attention's own bar for its gradients (relative RMS 2e-2) holds behind the norm, too
    for got, leaf in ((grad[:, :, 0], leaves[0]), (grad[:, :, 1], leaves[1]), (dqw, leaves[2]), (dkw, leaves[3])):
        err = (got.double() - leaf.grad).norm() / leaf.grad.norm()
        assert err < 2e-2, err


def test_places_beyond_32_bits():
    """Rows whose elements lie behind 2^31 of their buffers, as slices of fused rows and one head behind the other."""
    S, hq, hk, d = 120000, 96, 24, 128
    qkv = torch.empty((1, S, hq + 2 * hk, d), dtype=torch.bfloat16, device=DEV)
    assert qkv.numel() > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(1)
    for x in qkv[0].split(20000):
        x.normal_(generator=g)
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    f = attn.rotary_frequencies(d)
    rope, w = attn.Rotary(f), (1 + 0.3 * torch.randn((2, d), generator=g, device=DEV)).bfloat16()
    pos = torch.arange(S, device=DEV, dtype=torch.int32)[None]
    out = torch.empty((1, hq, S, d), dtype=torch.bfloat16, device=DEV)
    a, b = attn.qk_norm_rope(q, k, rope, pos, w[0], w[1], q_out=out.transpose(1, 2))
    rows = torch.tensor([0, 1, 777, 59999, 87381, 87382, 119998, 119999], device=DEV)
    for got, x, ww in ((a, q, w[0]), (b, k, w[1])):
        check(got[:, rows], *ref.forward(x[:, rows], ww, pos[:, rows], f, False, 1.0, 1e-6), "rows")
    # the gradient, written over its operand
    attn.qk_norm_rope_backward(a, b, q, k, rope, pos, w[0], w[1], dq=a, dk=b)
    again = attn.qk_norm_rope(q[:, rows].contiguous(), k[:, rows].contiguous(), rope, pos[:, rows].contiguous(), w[0], w[1])
    for got, dy, x, ww in ((a, again[0], q, w[0]), (b, again[1], k, w[1])):
        dx, tol, _, _ = ref.backward(dy, x[:, rows], ww, pos[:, rows], f, False, 1.0, 1e-6, 1)
        check(got[:, rows], dx, tol, "gradient")
