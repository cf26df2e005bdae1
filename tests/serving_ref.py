"""64-bit references of the serving calls, from their definitions, and the
error bounds their tests use.

Bounds.  u is half a step of the output type, relative (bf16 2^-8, fp16 2^-11).
For a row with probabilities p, values v and query q:

  O: the probabilities enter the P.V product rounded to the 16-bit type (an
     error of u * sum p |v|), the result is rounded once (u * |O|), and an error
     dx of the logits shifts every p by a relative 2 dx at most.
  dx: D products summed in fp32 (an error of D * 2^-23 * sum |q||k| * scale,
     which allows for truncating adders) and three more fp32 operations.
  LSE: dx, a sum of n terms (n * 2^-24 relative), and 2^-21 for exp2 and log2.
"""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
GROUP = 64


def logit_error(D, reach):
    """dx for logits whose products sum to `reach` in absolute value."""
    return (D + 3) * 2.0 ** -23 * reach + 2.0 ** -22


def varlen(q, k, v, starts, scale, causal):
    """(o, lse, tolerance of o, tolerance of lse) of packed prompts, in float64; rows of no sequence are NaN."""
    total, hq, d = q.shape
    g = hq // k.shape[1]
    o = torch.full((total, hq, d), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.full_like(o, math.nan)
    lse = torch.full((hq, total), math.nan, dtype=torch.float64, device=q.device)
    lse_tol = torch.full_like(lse, math.nan)
    u = HALF_STEP[q.dtype]
    for a, b in zip(starts, starts[1:]):
        if b <= a:
            continue
        for h in range(hq):
            qq, kk, vv = q[a:b, h].double(), k[a:b, h // g].double(), v[a:b, h // g].double()
            x = qq @ kk.T * scale
            reach = (qq.abs() @ kk.abs().T * scale).amax(1)
            if causal:
                x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(1), -math.inf)
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            o[a:b, h], lse[h, a:b] = p @ vv, z
            dx = logit_error(d, reach)
            mean = p @ vv.abs()
            tol[a:b, h] = u * (mean + o[a:b, h].abs()) + (2 * dx[:, None] + (b - a) * 2.0 ** -23) * mean + 1e-7
            lse_tol[h, a:b] = dx + (b - a) * 2.0 ** -24 + 2.0 ** -21
    return o, lse, tol, lse_tol


def quantise(x):
    """(codes, s, m) of rows x [..., D] in the cache's format, in float64."""
    y = x.double().unflatten(-1, (-1, GROUP))
    low, high = y.amin(-1), y.amax(-1)
    m = low.bfloat16().double()
    s = ((high - low) / 15).bfloat16().double()
    c = torch.round((y - m[..., None]) / s[..., None].where(s[..., None] != 0, torch.ones_like(s[..., None])))
    c = c.clamp(0, 15).where(s[..., None] != 0, torch.zeros_like(c))
    return c.flatten(-2), s, m


def pack(c):
    c = c.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()


def values(codes, meta):
    """Values that codes [..., D/2] with meta [..., D/64, 2] stand for, in float64."""
    sm = meta.double().repeat_interleave(GROUP, dim=-2)
    return unpack(codes) * sm[..., 0] + sm[..., 1]


def decode(q, cache, lens, scale):
    """(o, lse, weights [B, H, cap], tolerances of the three) of one token per sequence, in float64."""
    B, hq, d = q.shape
    H, cap = cache.H_kv, cache.capacity
    g = hq // H
    u = HALF_STEP[q.dtype]
    # p * s enters P.V in fp16, whatever the type: half a step of 11 bits
    up = 2.0 ** -11
    o = torch.zeros((B, hq, d), dtype=torch.float64, device=q.device)
    tol, lse = torch.zeros_like(o), torch.full((B, hq), -math.inf, dtype=torch.float64, device=q.device)
    lse_tol = torch.zeros_like(lse)
    w = torch.zeros((B, H, cap), dtype=torch.float64, device=q.device)
    w_tol = torch.zeros_like(w)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        if n == 0:
            continue
        for h in range(H):
            sm = [cache.k_meta[b, h, :n].double().repeat_interleave(GROUP, -2), cache.v_meta[b, h, :n].double().repeat_interleave(GROUP, -2)]
            c = [unpack(cache.k_codes[b, h, :n]), unpack(cache.v_codes[b, h, :n])]
            k, v = (c[i] * sm[i][..., 0] + sm[i][..., 1] for i in (0, 1))
            # the calls split a key into s c and m, a value into s (c - 8) and m + 8 s
            k_abs, v_part, v_off = (sm[0][..., 0] * c[0] + sm[0][..., 1].abs(),
                                    (sm[1][..., 0] * (c[1] - 8)).abs(), (sm[1][..., 1] + 8 * sm[1][..., 0]).abs())
            qq = q[b, h * g:(h + 1) * g].double()
            x = qq @ k.T * scale
            dx = logit_error(d, (qq.abs() @ k_abs.T * scale).amax(1))
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            o[b, h * g:(h + 1) * g] = p @ v
            lse[b, h * g:(h + 1) * g] = z
            lse_tol[b, h * g:(h + 1) * g] = dx + n * 2.0 ** -24 + 2.0 ** -21
            tol[b, h * g:(h + 1) * g] = (up * (p @ v_part) + u * (p @ v).abs() + (2 * dx[:, None] + n * 2.0 ** -23) * (p @ (v_part + v_off))
                                         + 1e-7)
            w[b, h, :n] = p.sum(0)
            w_tol[b, h, :n] = (p * (2 * dx[:, None] + n * 2.0 ** -23 + g * 2.0 ** -24)).sum(0) + 1e-30
    return o, lse, w, tol, lse_tol, w_tol


def evict(weight, pos, n, budget, recent):
    """Slots whose entries make up one (sequence, key head) after an eviction, in slot order: lists of numbers in and out."""
    if n <= budget:
        return list(range(n))
    newest = max(pos[:n])

    def rank(j):
        if pos[j] > newest - recent:
            return (0, 0.0, j)
        return (1, -math.inf, j) if math.isnan(weight[j]) else (2, -weight[j], j)

    kept = sorted(sorted(range(n), key=rank)[:budget])
    holes = sorted(set(range(budget)) - set(kept))
    src = list(range(budget))
    for hole, far in zip(holes, [j for j in kept if j >= budget]):
        src[hole] = far
    return src
