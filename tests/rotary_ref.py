"""64-bit references of the head norm with the rotation by position, and of the
calls on a paged cache, from their definitions, with the bounds their tests use.

Bounds.  u is half a step of the output type, relative; e32 = 2^-24.  An fp16
result below 2^-14 is off by 2^-25 at most.

  r = 1 / sqrt(mean(x^2) + eps): a sum of D squares (D e32, and 2 e32 each for the
     scaling and eps), halved by the root, and 2 ulp (4 e32) for rsqrt: within
     (D + 8) e32, relative.
  cos, sin: the angle's 24-bit number of half turns is off by 2^-25 of at most 1
     (times pi), sincospif by 2 ulp: within 2^-22, and the amplitude's product e32.
  Forward: two products and a sum of normed channels a, b:
     u |y| + ((D + 8) e32 + 2^-22 + 6 e32) amp (|a| + |b|).
  Gradient: g as the forward's turn; then r (g w - x r^2 mean(g w x)): the mean is a
     sum of D products (D e32) and r enters it three times:
     u |dx| + (4 (D + 8) e32 + 2^-22 + 16 e32) r (G w + |x^| mean(G w |x^|)), G being
     |a| + |b| of dy's pair.
  Weights' gradients: each term within ((D + 8) e32 + 2^-22 + 8 e32) G |x^|, and sums
     of n of them in a chain of fp32 additions n e32 more; the chains are a lane's
     (its rows) and a block's (8 warps, 5 exchanges).
"""
from __future__ import annotations

import math

import torch

from tests.serving_ref import HALF_STEP, logit_error

E32 = 2.0 ** -24
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def turn(x, pos, freqs, inter, amp, back=False):
    """x [..., H, D] float64 turned by pos [...]."""
    rot = 2 * len(freqs)
    if rot == 0:
        return x.clone()
    t = pos.double()[..., None, None] * torch.tensor(freqs, dtype=torch.float64, device=x.device)
    c, s = torch.cos(t) * amp, torch.sin(t) * amp
    if back:
        s = -s
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * c - b * s, a * s + b * c
    return y


def reach(x, freqs, inter, amp):
    """amp * (|a| + |b|) of each channel's pair; |x| where it is not turned."""
    rot = 2 * len(freqs)
    y = x.abs().clone()
    if inter:
        both = (y[..., 0:rot:2] + y[..., 1:rot:2]) * abs(amp)
        y[..., 0:rot:2] = both
        y[..., 1:rot:2] = both
    else:
        both = (y[..., :rot // 2] + y[..., rot // 2:rot]) * abs(amp)
        y[..., :rot] = torch.cat([both, both], -1)
    return y


def forward(x, w, pos, freqs, inter, amp, eps):
    """(y, tolerance) of one of q and k."""
    D = x.shape[-1]
    z = x.double()
    if w is not None:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * w.double()
    y = turn(z, pos, freqs, inter, amp)
    tol = HALF_STEP[x.dtype] * y.abs() + ((D + 14) * E32 + 2.0 ** -22) * reach(z, freqs, inter, amp) + TINY[x.dtype]
    return y, tol


def backward(dy, x, w, pos, freqs, inter, amp, eps, chain):
    """(dx, tolerance, dw, tolerance): the last two None without a norm."""
    D = x.shape[-1]
    u = HALF_STEP[x.dtype]
    g = turn(dy.double(), pos, freqs, inter, amp, back=True)
    G = reach(dy.double(), freqs, inter, amp)
    if w is None:
        return g, u * g.abs() + (2.0 ** -22 + 6 * E32) * G + TINY[x.dtype], None, None
    z, ww = x.double(), w.double()
    r = 1 / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
    hat = z * r
    dx = r * (g * ww - hat * (g * ww * hat).mean(-1, keepdim=True))
    size = r * (G * ww.abs() + hat.abs() * (G * ww.abs() * hat.abs()).mean(-1, keepdim=True))
    tol = u * dx.abs() + (4 * (D + 8) * E32 + 2.0 ** -22 + 16 * E32) * size + TINY[x.dtype]
    dw = (g * hat).flatten(0, -2).sum(0)
    dw_tol = ((D + 16 + chain + 13) * E32 + 2.0 ** -22) * (G * hat.abs()).flatten(0, -2).sum(0)
    return dx, tol, dw, dw_tol


def gather(pages, table, n, n_pages):
    """Entries 0 .. n - 1 of a sequence, [n, H, D] float64; zeros where the table names no page."""
    page = pages.shape[2]
    j = torch.arange(n, device=pages.device)
    at = table.long()[j // page]
    there = (at >= 0) & (at < n_pages)
    x = pages[at.clamp(0, n_pages - 1), :, j % page].double()
    return torch.where(there[:, None, None], x, 0.0)


def attend(q, k_pages, v_pages, table, length, starts, scale, window=None, sinks=0, max_len=None, max_new=None):
    """(o, lse, tolerances) of new tokens over a paged cache: q [rows, H_q, D]; starts None: a token each.
    Rows of no sequence are NaN.  Bounds as those of packed prompts: P enters P V in the 16-bit type."""
    rows, hq, d = q.shape
    H, cap = k_pages.shape[1], table.shape[1] * k_pages.shape[2]
    g = hq // H
    u = HALF_STEP[q.dtype]
    o = torch.full((rows, hq, d), math.nan, dtype=torch.float64, device=q.device)
    tol, lse = torch.full_like(o, math.nan), torch.full((rows, hq), math.nan, dtype=torch.float64, device=q.device)
    lse_tol = torch.full_like(lse, math.nan)
    if starts is None:
        starts = list(range(table.shape[0] + 1))
    starts = [min(max(x, 0), rows) for x in starts]
    for b, (a, e) in enumerate(zip(starts, starts[1:])):
        new = e - a
        if new <= 0:
            continue
        n = min(max(int(length[b]), 0), cap if max_len is None else min(cap, max_len))
        k, v = gather(k_pages, table[b], n, k_pages.shape[0]), gather(v_pages, table[b], n, k_pages.shape[0])
        pos = torch.arange(n - new, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)
        seen = j <= pos
        if window is not None:
            seen &= (j > pos - window) | (j < sinks)
        done = new if max_new is None else min(new, max_new)
        for h in range(hq):
            qq, kk, vv = q[a:e, h].double(), k[:, h // g], v[:, h // g]
            x = (qq @ kk.T * scale).masked_fill(~seen, -math.inf)
            far = (qq.abs() @ kk.abs().T * scale).masked_fill(~seen, 0.0).amax(1) if n else torch.zeros(new, dtype=torch.float64, device=q.device)
            z = torch.logsumexp(x, 1) if n else torch.full((new,), -math.inf, dtype=torch.float64, device=q.device)
            p = torch.exp(x - z.where(z > -math.inf, torch.zeros_like(z))[:, None])
            dx = logit_error(d, far)
            # masked V may be anything: it has no part
            vv_abs = vv.abs()
            y, mean = p @ vv, p @ vv_abs
            s = slice(a, a + done)
            o[s, h], lse[s, h] = y[:done], z[:done]
            tol[s, h] = (u * (mean + y.abs()) + (2 * dx[:, None] + n * 2.0 ** -23) * mean + 1e-7)[:done]
            lse_tol[s, h] = (dx + n * 2.0 ** -24 + 2.0 ** -21)[:done]
    return o, lse, tol, lse_tol
