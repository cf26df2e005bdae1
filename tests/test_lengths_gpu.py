"""Lengths that an append writes and the attention behind it reads, where old lengths,
new ones, starts and the page table lie side by side in one small buffer: every step
sees the lengths of its own append, call by call and replayed from a graph, where the
attention's blocks are on the GPU before the append has ended."""
from __future__ import annotations

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn

pytestmark = pytest.mark.gpu

DEV = "cuda"


def captured(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    return graph, held


def same(got, want):
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]), f"step {i}"


@pytest.mark.parametrize("new", [1, 3, 20])  # 8 and 16 rows a key head in the token kernel; chunks, with a list where long
@pytest.mark.parametrize("B,long", [(3, False), (3, True), (24, False)])
def test_pages(B, long, new):
    H, hq, d, page, turns = 2, 8, 64, 16, 24
    had = 3000 if long else 40
    pages = -(-(had + turns * new) // page)
    apart = attn.PagedKVCache.empty(B, H, B * pages, page, pages, d)
    apart.page_table.copy_(torch.randperm(B * pages, device=DEV).int().view(B, pages))
    g = torch.Generator(device=DEV).manual_seed(new)
    apart.k_pages.normal_(generator=g)
    apart.v_pages.normal_(generator=g)
    apart.length.fill_(had)
    starts = (torch.arange(B + 1, device=DEV) * new).int()
    # one buffer: lengths in turn, starts, the table
    ints = torch.zeros(3 * B + 1 + B * pages, dtype=torch.int32, device=DEV)
    pair, s, table = ints[:2 * B].view(2, B), ints[2 * B:3 * B + 1], ints[3 * B + 1:].view(B, pages)
    s.copy_(starts)
    table.copy_(apart.page_table)
    pair[0].fill_(had)
    beside = attn.PagedKVCache(apart.k_pages.clone(), apart.v_pages.clone(), table, pair[0])
    first = beside.k_pages.clone(), beside.v_pages.clone()
    qkv = torch.randn((turns, B * new, hq + 2 * H, d), generator=g, device=DEV).bfloat16()

    def step(c, i, seq_start, out=None):
        q, k, v = qkv[i, :, :hq], qkv[i, :, hq:hq + H], qkv[i, :, hq + H:]
        q = c.append(k, v, seq_start=seq_start, q=q, length_out=out)
        if out is not None:
            c.length = out
        return c.attend(q, seq_start, max_new=new)

    want = []
    for i in range(turns):
        want.append(step(apart, i, starts))
        torch.cuda.synchronize()

    def all_steps():
        beside.length = pair[0]
        return [step(beside, i, s, pair[1 - i % 2]) for i in range(turns)]

    def reset():
        beside.k_pages.copy_(first[0])
        beside.v_pages.copy_(first[1])
        pair.zero_()
        pair[0].fill_(had)

    got = all_steps()
    torch.cuda.synchronize()
    same(got, want)
    graph, held = captured(all_steps)
    for _ in range(5):
        reset()
        for o, lse in held:
            o.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(held, want)
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    assert (pair[turns % 2] == had + turns * new).all()
