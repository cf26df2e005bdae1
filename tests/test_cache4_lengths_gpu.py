"""The 4-bit cache with its old and new lengths side by side in one buffer: every step's
attention sees the lengths of its own append, call by call and replayed from a graph."""
from __future__ import annotations

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests.test_lengths_gpu import DEV, captured, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("B,long", [(3, False), (3, True), (24, False), (300, False)])
def test_steps(B, long, weights):
    H, hq, d, turns = 2, 8, 64, 24
    had = 3000 if long else 40
    apart = attn.KVCache4.empty(B, H, had + turns + 4, d)
    g = torch.Generator(device=DEV).manual_seed(B)
    fill = torch.randn((B * had, 2 * H, d), generator=g, device=DEV).bfloat16()
    apart.append(fill[:, :H], fill[:, H:], seq_start=(torch.arange(B + 1, device=DEV) * had).int())
    pair = torch.zeros((2, B), dtype=torch.int32, device=DEV)
    pair[0].fill_(had)
    names = ("k_codes", "k_meta", "v_codes", "v_meta", "weight", "pos")
    beside = attn.KVCache4(*(getattr(apart, n).clone() for n in names), pair[0])
    first = [getattr(apart, n).clone() for n in names]
    qkv = torch.randn((turns, B, hq + 2 * H, d), generator=g, device=DEV).bfloat16()

    def step(c, i, out=None):
        c.append(qkv[i, :, hq:hq + H], qkv[i, :, hq + H:], length_out=out)
        if out is not None:
            c.length = out
        return c.attend(qkv[i, :, :hq], weight_out=torch.empty_like(c.weight) if weights else None)

    want = []
    for i in range(turns):
        want.append(step(apart, i))
        torch.cuda.synchronize()

    def all_steps():
        beside.length = pair[0]
        return [step(beside, i, pair[1 - i % 2]) for i in range(turns)]

    got = all_steps()
    torch.cuda.synchronize()
    same(got, want)
    graph, held = captured(all_steps)
    for _ in range(5):
        for n, x in zip(names, first):
            getattr(beside, n).copy_(x)
        pair.zero_()
        pair[0].fill_(had)
        for o, lse in held:
            o.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(held, want)
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
