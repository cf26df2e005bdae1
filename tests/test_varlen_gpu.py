"""attn_fwd_varlen against the 64-bit definition: lengths, grouped heads,
types, strides, what lies outside the sequences, streams and graphs."""
from __future__ import annotations

import math

import pytest
import torch

import io_aware_attention_fwd_gb300 as attn
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu


def make(lens, hq, hkv, d, dtype, pad=0, seed=0, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = sum(lens) + pad
    if fused:
        x = torch.randn((total, hq + 2 * hkv, d), generator=g, device="cuda").to(dtype)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (torch.randn((total, h, d), generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    return q, k, v, starts, torch.tensor(starts, dtype=torch.int32, device="cuda")


def check(got, want):
    o, lse = got
    ro, rlse, tol, lse_tol = want
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK
    own = ~rlse.isnan()
    assert ((lse.double() - rlse).abs() <= lse_tol)[own].all(), (lse.double() - rlse).abs()[own].max()
    own = ~ro.isnan()
    bad = ((o.double() - ro).abs() > tol)[own]
    assert not bad.any(), (int(bad.sum()), (o.double() - ro).abs()[own].max())


LENGTHS = [
    [1], [2, 1, 1], [127], [128], [129], [64, 0, 65, 0, 0, 1], [0, 0, 300], [255, 256, 257], [513, 3, 1000],
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_lengths(lens, d, causal):
    q, k, v, starts, s = make(lens, 8, 2, d, torch.bfloat16, seed=len(lens))
    scale = 1 / math.sqrt(d)
    check(attn.attention_varlen(q, k, v, s, causal=causal), ref.varlen(q, k, v, starts, scale, causal))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (6, 3), (3, 1), (5, 1), (14, 2), (16, 2), (12, 1), (48, 2), (100, 1), (128, 1)])
def test_groups(hq, hkv, dtype):
    q, k, v, starts, s = make([37, 200, 1], hq, hkv, 64, dtype, seed=hq)
    check(attn.attention_varlen(q, k, v, s), ref.varlen(q, k, v, starts, 0.125, True))
    q, k, v, starts, s = make([70, 9], hq, hkv, 128, dtype, seed=hq)
    check(attn.attention_varlen(q, k, v, s, scale=0.2, causal=False), ref.varlen(q, k, v, starts, 0.2, False))


@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences(d):
    """More sequences than the listing block has warps, more units than SMs, units of equal and of unlike weight."""
    lens = [(i * 37) % 150 for i in range(400)] + [700]
    q, k, v, starts, s = make(lens, 4, 2, d, torch.bfloat16, seed=5)
    check(attn.attention_varlen(q, k, v, s), ref.varlen(q, k, v, starts, 1 / math.sqrt(d), True))


def test_long_prompt_sampled_rows():
    q, k, v, starts, s = make([9000], 8, 2, 128, torch.bfloat16, seed=6)
    o, lse = attn.attention_varlen(q, k, v, s)
    ro, rlse, tol, lse_tol = ref.varlen(q, k, v, starts, 128 ** -0.5, True)
    check((o, lse), (ro, rlse, tol, lse_tol))


def test_contiguous_and_fused_inputs_agree():
    q, k, v, starts, s = make([300, 45], 8, 4, 64, torch.bfloat16)
    a = attn.attention_varlen(q, k, v, s)
    b = attn.attention_varlen(q.contiguous(), k.contiguous(), v.contiguous(), s)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal", [True, False])
def test_nothing_outside_a_sequence_reaches_it(causal, value):
    """Rows behind the last sequence, and neighbours, hold NaN or infinities: no effect; padding rows are not written."""
    lens, pad = [100, 30, 129], 77
    q, k, v, starts, s = make(lens, 8, 2, 128, torch.bfloat16, pad=pad, seed=1, fused=False)
    want = ref.varlen(q, k, v, starts, 128 ** -0.5, causal)
    for x in (q, k, v):
        x[259:] = value
        x[100:130] = value
    out = torch.full_like(q, 7.0).contiguous()
    lse = torch.full((8, q.shape[0]), 7.0, device="cuda")
    o, z = attn.attention_varlen(q, k, v, s, causal=causal, out=out, lse=lse)
    assert o is out and z is lse
    torch.cuda.synchronize()
    assert (out[259:] == 7.0).all() and (lse[:, 259:] == 7.0).all()
    keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    keep[100:130] = False
    keep[259:] = False
    nan = torch.full_like
    check((out, lse), tuple(torch.where(keep[:, None, None] if x.dim() == 3 else keep, x, nan(x, math.nan)) for x in want))


def test_gap_before_the_first_sequence():
    q, k, v, _, _ = make([50], 4, 4, 64, torch.bfloat16, fused=False)
    s = torch.tensor([10, 40, 40, 45], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    o, lse = attn.attention_varlen(q, k, v, s, out=out)
    ro, rlse, tol, lse_tol = ref.varlen(q, k, v, [10, 40, 40, 45], 0.125, True)
    check((o, lse), (ro, rlse, tol, lse_tol))
    assert (out[:10] == 3.0).all() and (out[45:] == 3.0).all()


def test_starts_out_of_range_are_clamped():
    q, k, v, _, _ = make([64], 4, 4, 64, torch.bfloat16, fused=False)
    s = torch.tensor([-5, 20, 2000], dtype=torch.int32, device="cuda")
    o, lse = attn.attention_varlen(q, k, v, s)
    check((o, lse), ref.varlen(q, k, v, [0, 20, 64], 0.125, True))


def test_large_logits():
    """Logits that grow along the keys: the running maximum moves many times."""
    q, k, v, starts, s = make([700, 300], 4, 2, 64, torch.bfloat16, seed=9, fused=False)
    k *= torch.linspace(0.1, 12, k.shape[0], device="cuda")[:, None, None].bfloat16()
    check(attn.attention_varlen(q, k, v, s, scale=0.5), ref.varlen(q, k, v, starts, 0.5, True))


def test_matches_the_dense_call():
    """Equal lengths and as many key as query heads: attention_forward's result (both within their bounds of each other)."""
    B, H, S, D = 3, 4, 320, 128
    q, k, v, starts, s = make([S] * B, H, H, D, torch.bfloat16, fused=False)
    o, lse = attn.attention_varlen(q, k, v, s)
    dense = [x.reshape(B, S, H, D).transpose(1, 2).contiguous() for x in (q, k, v)]
    od, ld = attn.attention_forward(*dense, causal=True, n_splits=1)
    _, _, tol, lse_tol = ref.varlen(q, k, v, starts, D ** -0.5, True)
    assert ((o.double() - od.transpose(1, 2).reshape(B * S, H, D).double()).abs() <= 2 * tol).all()
    assert ((lse.double() - ld.transpose(0, 1).reshape(H, B * S).double()).abs() <= 2 * lse_tol).all()


def test_side_stream_and_two_graphs():
    q, k, v, starts, s = make([150, 40, 300], 8, 2, 64, torch.bfloat16, seed=2)
    want = attn.attention_varlen(q, k, v, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = attn.attention_varlen(q, k, v, s, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    outs, graphs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(attn.attention_varlen(q, k, v, s))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # the lengths are read from the device at every replay
    s.copy_(torch.tensor([0, 20, 400, 490], dtype=torch.int32))
    graphs[0].replay()
    check(outs[0], ref.varlen(q, k, v, [0, 20, 400, 490], 0.125, True))


def test_results_do_not_change_from_call_to_call():
    q, k, v, starts, s = make([1500, 1, 700, 64, 64, 64], 16, 4, 128, torch.float16, seed=4)
    a = attn.attention_varlen(q, k, v, s)
    for _ in range(3):
        b = attn.attention_varlen(q, k, v, s)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_no_rows():
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = attn.attention_varlen(q, q, q, s)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    # rows, but every sequence empty
    q, k, v, _, _ = make([10], 4, 4, 64, torch.bfloat16, fused=False)
    out = torch.full_like(q, 2.0)
    attn.attention_varlen(q, k, v, s, out=out)
    torch.cuda.synchronize()
    assert attn.attn_fwd_debug_status() == attn.ATTN_OK and (out == 2.0).all()
