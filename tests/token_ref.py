"""Attention of few rows a key head (PagedKVCache.attend up to 16 of them) in 64 bits, with
the bound of a kernel that holds P in two 16-bit terms.

u is half a step of the 16-bit type, relative.  Of O, relative to mean = sum p |v|:
  u |O|               the result's rounding;
  u^2                 P: hi = x (1 + u), lo takes up x - hi to u of it.  fp16 holds P 2^11
                      times as large and not below 2^-24: lo is off by 2^-25 at most, which of
                      a row's 2^11 is 2^-36 |v| a key;
  2 (dx + 2^-21)      the logits, above and below the division; exponents up to 16 have half
                      a step of 2^-21 in fp32;
  (3 n + 64) 2^-23    sums: n products of hi, n of lo and n of P one behind the other, the
                      tensor core's truncated, then the warps', the shares' and the division.
LSE: dx + n 2^-24 + 2^-21."""
from __future__ import annotations

import math

import torch

from tests.serving_ref import HALF_STEP, logit_error

TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def attend(q, k, v, dtype, scale, once=False):
    """(o, lse, tolerances) of q [rows, D] over k, v [n, D] that all rows see, float64.  once: with
    P rounded to the 16-bit type and no second term, as a kernel would that drops it."""
    n, d = k.shape
    u = HALF_STEP[dtype]
    x = q @ k.T * scale
    dx = logit_error(d, (q.abs() @ k.abs().T * scale).amax(1))[:, None]
    z = torch.logsumexp(x, 1)
    p = torch.exp(x - z[:, None])
    mean = p @ v.abs()
    w = p
    if once:
        up = 2.0 ** 11 if dtype == torch.float16 else 1.0
        top = p.amax(1, keepdim=True)
        w = (p / top * up).to(dtype).double() / up * top
    o = w @ v
    tol = u * (p @ v).abs() + (u * u + 2 * (dx + 2.0 ** -21) + (3 * n + 64) * 2.0 ** -23) * mean + TINY[dtype]
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -36 * v.abs().amax(0)
    return o, z, tol, dx[:, 0] + n * 2.0 ** -24 + 2.0 ** -21


def make(n, rows, d, dtype, seed, device="cpu"):
    """Small logits, so that their own error hides nothing: q, k, v of one key head, in the 16-bit type."""
    g = torch.Generator(device=device).manual_seed(seed)
    q = torch.randn((rows, d), generator=g, device=device) / 16
    k, v = torch.randn((2, n, d), generator=g, device=device)
    return q.to(dtype), k.to(dtype), v.to(dtype)
