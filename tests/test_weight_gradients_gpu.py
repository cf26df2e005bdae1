"""Gradients of the norm weights over many rows: long chains of fp32 additions, terms of
one sign as well as of both, against sums in 64 bits."""
from __future__ import annotations

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import rotary_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def chain(B, S, hq, hk, d):
    """Rows of one lane: the list of all tokens' groups of heads is cut into 152 * 2 * 8 equal shares, one a warp."""
    rows = 32 // (d // 8)
    groups = -(-hq // rows) + -(-hk // rows)
    return -(-B * S * groups // (152 * 2 * 8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,S,hq,hk,d,rot,inter", [(2, 8192, 32, 8, 128, 96, True), (1, 20000, 14, 2, 64, 64, False), (3, 9001, 8, 8, 64, 16, False)])
@pytest.mark.parametrize("mean", [0.0, 1.0])
def test_many_rows(mean, B, S, hq, hk, d, rot, inter, dtype):
    g = torch.Generator(device=DEV).manual_seed(S)
    f = attn.rotary_frequencies(rot)
    rope = attn.Rotary(f, interleaved=inter, amplitude=1.2)
    pos = torch.arange(S, device=DEV, dtype=torch.int32).expand(B, S).contiguous()
    w = list((1 + 0.3 * torch.randn((2, d), generator=g, device=DEV)).to(dtype))
    q, k = ((torch.randn((B, S, h, d), generator=g, device=DEV) + mean).to(dtype) for h in (hq, hk))
    dq, dk = ((torch.randn((B, S, h, d), generator=g, device=DEV) + mean).to(dtype) for h in (hq, hk))
    got = attn.qk_norm_rope_backward(dq, dk, q, k, rope, pos, *w)
    torch.cuda.synchronize()
    n = chain(B, S, hq, hk, d)
    for x, dy, ww, grad, dw in ((q, dq, w[0], got[0], got[2]), (k, dk, w[1], got[1], got[3])):
        total, tol = torch.zeros(d, dtype=torch.float64, device=DEV), torch.zeros(d, dtype=torch.float64, device=DEV)
        for b in range(B):  # (a batch and 4096 rows at a time, for the memory)
            for r in range(0, S, 4096):
                at = (slice(b, b + 1), slice(r, r + 4096))
                dx, dx_tol, part, part_tol = ref.backward(dy[at], x[at], ww, pos[at], f, inter, 1.2, 1e-6, n)
                assert ((grad[at].double() - dx).abs() <= dx_tol).all()
                total += part
                tol += part_tol
        assert ((dw.double() - total).abs() <= tol).all(), ((dw.double() - total).abs() / tol).max()


def test_the_workspace_is_what_the_grid_writes():
    """Two blocks an SM at most, each a row of fp32 [2][D]."""
    for args in ((1, 1, 1, 1, 64), (1, 100, 32, 8, 128), (2, 8192, 32, 8, 128), (1, 1 << 22, 96, 24, 64)):
        n = attn.attn_qk_norm_rope_bwd_workspace_bytes(*args)
        assert 0 < n <= 152 * 2 * 2 * args[-1] * 4 and n % (2 * args[-1] * 4) == 0
