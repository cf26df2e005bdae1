"""Cases of the position rotation and the paged K/V cache, for measuring them.

Three operators that stand around attention, in the order a token meets them:

  rotate   the norm of every query and key head and the rotation by its
           position, in one pass, and its gradient (qk_norm_rope,
           qk_norm_rope_backward)
  write    the same on a step's new tokens, with the keys and values written
           into the pages of a cache (PagedKVCache.append)
  attend   attention of the new tokens, one of each sequence or a chunk, over
           the pages, with or without a sliding window and first tokens that
           stay visible (PagedKVCache.attend)

A head's D channels are normed as x / sqrt(mean(x^2) + eps) * weight; of the
result the first R channels are turned: pair i by position * f[i], where pair i
is channels (i, i + R/2) or, interleaved, (2i, 2i + 1), times an amplitude.
Sequence b's entry j lies in row j % page of page table[b, j // page].  Of its n
newest entries, which have queries, the i-th has position length - n + i and
sees entry j if j <= position and (there is no window, or j > position - window,
or j < sinks).
"""
import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --- cases -----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the new tokens of 64 running sequences, somewhere in a long context: latency
        dict(name="rotate_token", op="rotate", back=False, b=1, s=64, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, amp=1.0, far=131072,
             type="bf16"),
        # a training step's queries and keys, from the projection's rows to heads one behind the other
        dict(name="rotate_dense", op="rotate", back=False, b=2, s=8192, hq=32, hkv=32, d=128, rot=128, inter=False, norm=True, amp=1.0, far=0,
             type="bf16"),
        # its gradient, grouped heads, three quarters of a head turned
        dict(name="rotate_back", op="rotate", back=True, b=2, s=8192, hq=32, hkv=8, d=128, rot=96, inter=True, norm=True, amp=1.2, far=0, type="bf16"),
        # the new token of every running sequence into its page
        dict(name="write_token", op="write", n=64, longest=1, pad=0, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, amp=1.0, page=64, ctx=4000,
             type="bf16", lens=21),
        # a prefill batch's keys and values, small pages
        dict(name="write_prompt", op="write", n=12, longest=5000, pad=21, hq=32, hkv=8, d=128, rot=64, inter=False, norm=True, amp=1.0, page=16,
             ctx=3000, type="bf16", lens=22),
        # one user, short history, as many key as query heads: latency
        dict(name="token_short", op="attend", n=1, new=1, pad=0, ctx=700, equal=True, hq=16, hkv=16, d=64, page=16, window=0, sinks=0, type="fp16",
             lens=0),
        # one user, very long history
        dict(name="token_long", op="attend", n=1, new=1, pad=0, ctx=131071, equal=True, hq=32, hkv=8, d=128, page=64, window=0, sinks=0, type="bf16",
             lens=0),
        # a full batch of long histories, eight query heads to a key head
        dict(name="token_full", op="attend", n=64, new=1, pad=0, ctx=15999, equal=False, hq=64, hkv=8, d=128, page=64, window=0, sinks=0, type="bf16",
             lens=23),
        # a batch that attends to its last 4096 tokens and four first ones
        dict(name="token_window", op="attend", n=32, new=1, pad=0, ctx=32767, equal=False, hq=32, hkv=8, d=128, page=16, window=4096, sinks=4,
             type="bf16", lens=24),
        # a user's next message over a long conversation
        dict(name="chunk_long", op="attend", n=1, new=512, pad=0, ctx=32256, equal=True, hq=32, hkv=8, d=128, page=64, window=0, sinks=0, type="bf16",
             lens=0),
        # a batch of messages of many lengths over histories of many lengths
        dict(name="chunk_batch", op="attend", n=16, new=301, pad=13, ctx=8000, equal=False, hq=32, hkv=8, d=128, page=32, window=0, sinks=0,
             type="bf16", lens=25),
        # one long document, each token attending to 4096 before it and 64 first ones
        dict(name="prompt_window", op="attend", n=1, new=16384, pad=0, ctx=0, equal=True, hq=32, hkv=8, d=128, page=128, window=4096, sinks=64,
             type="bf16", lens=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "write", "attend", "attend"])
    d, kind = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    turn = dict(rot=rng.choice([16 * i for i in range(1, d // 16 + 1)] + [d, d]), inter=rng.random() < 0.5, norm=rng.random() < 0.7,
                amp=rng.choice([1.0, 1.0, 1.2]))
    seed = rng.randrange(1, 1 << 30)
    while True:
        if op == "rotate":
            c = dict(op=op, back=rng.random() < 0.5, b=_log(rng, 1, 16), s=_log(rng, 1, 8192), hq=hq, hkv=hkv, d=d, **turn,
                     far=rng.choice([0, _log(rng, 1, 1000000)]), type=kind)
            if work(c)["bytes"] <= work(listed()[2])["bytes"]:
                return c
        elif op == "write":
            c = dict(op=op, n=_log(rng, 1, 64), longest=_log(rng, 1, 8000), pad=rng.choice([0, rng.randrange(1, 100)]), hq=hq, hkv=hkv, d=d, **turn,
                     page=rng.choice([16, 32, 64, 128, 256]), ctx=_log(rng, 1, 100000), type=kind, lens=seed)
            if c["longest"] == 1:
                c["pad"] = 0
            if work(c)["bytes"] <= work(listed()[4])["bytes"] and c["n"] * (c["ctx"] + c["longest"]) * hkv <= 1 << 22:
                return c
        else:
            one = rng.random() < 0.5
            c = dict(op=op, n=_log(rng, 1, 64), new=1 if one else _log(rng, 2, 8192), pad=0 if one else rng.choice([0, rng.randrange(1, 100)]),
                     ctx=rng.choice([0, _log(rng, 1, 131071), _log(rng, 1, 131071)]), equal=False, hq=hq, hkv=hkv, d=d,
                     page=rng.choice([16, 32, 64, 128, 256]), window=rng.choice([0, 0, _log(rng, 1, 32768)]), sinks=0, type=kind, lens=seed)
            if c["window"]:
                c["sinks"] = rng.choice([0, rng.randrange(1, 300)])
            t = sum(_lens(c)[1])
            rows = c["n"] * (c["ctx"] + c["new"])
            if t <= 16384 and rows * hkv * d <= 64 * 16000 * 8 * 128 and hq * t * (c["ctx"] + c["new"]) <= 32 * 16384 ** 2:
                w = work(c)
                if w["flops"] <= work(listed()[11])["flops"] and w["bytes"] <= work(listed()[7])["bytes"]:
                    return c


def _lens(c):
    """Entries that a case's sequences hold before the pass, and new ones: all equal where it says so, else spread, the first the longest, some of them empty or of one token."""
    n, new, ctx = c["n"], c.get("new", c.get("longest")), c["ctx"]
    if c.get("equal"):
        return [ctx] * n, [new] * n
    rng = random.Random(c["lens"])
    had, got = [ctx], [new]
    for _ in range(n - 1):
        u = rng.random()
        had.append(0 if u < 0.05 else max(0, int(ctx * rng.uniform(0.05, 1.0))))
        u = rng.random()
        got.append(new if new == 1 else 0 if u < 0.05 else 1 if u < 0.1 else max(1, int(new * rng.uniform(0.05, 1.0))))
    return had, got


def _frequencies(c):
    """Radians a position for each pair, in 64 bits: a base of 10000, slowed down fourfold where the amplitude says that the context was lengthened."""
    return [10000.0 ** (-2.0 * i / c["rot"]) / (4.0 if c["amp"] != 1.0 else 1.0) for i in range(c["rot"] // 2)]


# --- what a program has in hand --------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _starts(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _pages(g, c, lens, spare):
    """Pages of K and V and the table that says which a sequence has, in no order; places of the table that no entry needs name no page."""
    page = c["page"]
    need = [-(-x // page) for x in lens]
    count = sum(need) + spare
    kind = TYPES[c["type"]]
    k = torch.randn((count, c["hkv"], page, c["d"]), generator=g, device="cuda", dtype=kind)
    v = torch.randn((count, c["hkv"], page, c["d"]), generator=g, device="cuda", dtype=kind)
    k[..., 3::29] *= 2.0  # a few channels spread widely
    order = torch.randperm(count, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(1, max(need)) + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = order[at:at + x]
        at += x
    return k, v, table


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    kind, hq, hkv, d = TYPES[c["type"]], c["hq"], c["hkv"], c["d"]
    if c["op"] == "attend":
        had, got = _lens(c)
        rows = sum(got) + c["pad"]
        s["q"] = torch.randn((rows, hq, d), generator=g, device="cuda").to(kind)
        s["seq_start"] = None if c["new"] == 1 else _starts(got)
        length = [a + b for a, b in zip(had, got)]
        s["k_pages"], s["v_pages"], s["table"] = _pages(g, c, length, 3)
        s["length"] = torch.tensor(length, dtype=torch.int32, device="cuda")
        s["max_len"], s["max_new"] = max(1, max(length)), max(got)
        s["out"], s["lse"] = torch.zeros((rows, hq, d), dtype=kind, device="cuda"), torch.zeros((rows, hq), device="cuda")
    else:
        s["freq"] = _frequencies(c)
        if c["norm"]:
            s["qw"], s["kw"] = (1.0 + 0.2 * torch.randn((2, d), generator=g, device="cuda")).to(kind)
        else:
            s["qw"] = s["kw"] = None
        if c["op"] == "write":
            had, got = _lens(c)
            rows = sum(got) + c["pad"]
            shape = (rows,)
            s["seq_start"] = None if c["longest"] == 1 else _starts(got)
            s["length"] = torch.tensor(had, dtype=torch.int32, device="cuda")
            s["length_out"] = torch.zeros_like(s["length"])
            s["k_pages"], s["v_pages"], s["table"] = _pages(g, c, [a + b for a, b in zip(had, got)], 3)
            s["q_out"] = torch.zeros((rows, hq, d), dtype=kind, device="cuda")
        else:
            shape = (c["b"], c["s"])
            first = torch.randint(0, c["far"] + 1, (c["b"], 1), generator=g, device="cuda")
            s["pos"] = (first + torch.arange(c["s"], device="cuda")).int()
            if c["back"]:  # gradients as attention's backward pass leaves them
                s["dq"], s["dk"] = (torch.randn((c["b"], h, c["s"], d), generator=g, device="cuda").to(kind) for h in (hq, hkv))
        # q, k and v are slices of one projection's output
        qkv = torch.randn((*shape, hq + 2 * hkv, d), generator=g, device="cuda").to(kind)
        s["q"], s["k"], s["v"] = qkv[..., :hq, :], qkv[..., hq:hq + hkv, :], qkv[..., hq + hkv:, :]
        if own:
            from io_aware_attention_fwd_gb300 import Rotary
            s["rope"] = Rotary(s["freq"], interleaved=c["inter"], amplitude=c["amp"])
        else:
            s["freq"] = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    if own and c["op"] != "rotate":  # the framework's handle on these same buffers, which a program makes once
        from io_aware_attention_fwd_gb300 import PagedKVCache
        s["cache"] = PagedKVCache(s["k_pages"], s["v_pages"], s["table"], s["length"])
    return s


# --- one pass --------------------------------------------------------------------------------------------------------

def run(state):
    return {"rotate": _rotate, "write": _write, "attend": _attend}[state["case"]["op"]](state)


def _turn(s, pos):
    """Cosines and sines of positions [...], for every pair: [..., 1, R/2]."""
    angle = pos.double()[..., None, None] * s["freq"]
    amp = s["case"]["amp"]
    return (torch.cos(angle) * amp).float(), (torch.sin(angle) * amp).float()


def _pairs(x, c):
    """The two channels of every pair, and the channels that are not turned."""
    r = c["rot"]
    if c["inter"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _unpairs(a, b, rest, c):
    if c["inter"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _norm_turn(x, w, cos, sin, c):
    y = x.float()
    if w is not None:
        y = y * (1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)) * w.float()
    a, b, rest = _pairs(y, c)
    return _unpairs(a * cos - b * sin, a * sin + b * cos, rest, c).to(x.dtype)


def _norm_turn_back(dy, x, w, cos, sin, c):
    a, b, rest = _pairs(dy.float(), c)
    g = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, c)
    if w is None:
        return g.to(x.dtype), None
    x32 = x.float()
    r = 1.0 / torch.sqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    hat = x32 * r
    dw = (g * hat).flatten(0, -2).sum(0, dtype=torch.float64).float()
    gw = g * w.float()
    return (r * (gw - hat * (gw * hat).mean(-1, keepdim=True))).to(x.dtype), dw


def _rotate(s):
    c = s["case"]
    if own:
        from io_aware_attention_fwd_gb300 import qk_norm_rope, qk_norm_rope_backward
        if c["back"]:
            dq, dk, dqw, dkw = qk_norm_rope_backward(s["dq"].transpose(1, 2), s["dk"].transpose(1, 2), s["q"], s["k"], s["rope"], s["pos"],
                                                     q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
            return (dq, dk, dqw, dkw) if c["norm"] else (dq, dk)
        # attention takes [B, H, S, D]
        q, k = (torch.empty((c["b"], h, c["s"], c["d"]), dtype=s["q"].dtype, device="cuda") for h in (c["hq"], c["hkv"]))
        qk_norm_rope(s["q"], s["k"], s["rope"], s["pos"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, q_out=q.transpose(1, 2), k_out=k.transpose(1, 2))
        return q, k
    cos, sin = _turn(s, s["pos"])
    if not c["back"]:
        return tuple(_norm_turn(x, w, cos, sin, c).transpose(1, 2).contiguous() for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    dq, dqw = _norm_turn_back(s["dq"].transpose(1, 2), s["q"], s["qw"], cos, sin, c)
    dk, dkw = _norm_turn_back(s["dk"].transpose(1, 2), s["k"], s["kw"], cos, sin, c)
    return (dq, dk, dqw, dkw) if c["norm"] else (dq, dk)


def _places(s):
    """Of every real packed row: its number, its sequence and its entry."""
    at = torch.arange(s["q"].shape[0], device="cuda")
    if s["seq_start"] is None:
        return at, at, s["length"].long()
    seq = (at[:, None] >= s["seq_start"][None, 1:]).sum(1)
    real = (at < s["seq_start"][-1]).nonzero()[:, 0]
    seq = seq[real]
    return real, seq, real - s["seq_start"][seq] + s["length"][seq]


def _write(s):
    c = s["case"]
    if own:
        q = s["cache"].append(s["k"], s["v"], seq_start=s["seq_start"], q=s["q"], rope=s["rope"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                              q_out=s["q_out"], length_out=s["length_out"])
        return q, s["k_pages"], s["v_pages"], s["length_out"]
    real, seq, slot = _places(s)
    cos, sin = _turn(s, slot)
    q = s["q_out"].clone()
    q[real] = _norm_turn(s["q"][real], s["qw"], cos, sin, c)
    where, row = s["table"][seq, slot // c["page"]].long(), slot % c["page"]
    s["k_pages"][where, :, row] = _norm_turn(s["k"][real], s["kw"], cos, sin, c)
    s["v_pages"][where, :, row] = s["v"][real]
    new = 1 if s["seq_start"] is None else s["seq_start"][1:] - s["seq_start"][:-1]
    return q, s["k_pages"], s["v_pages"], s["length"] + new


def _attend(s):
    c = s["case"]
    if own:
        return s["cache"].attend(s["q"], seq_start=s["seq_start"], window=c["window"] or None, sinks=c["sinks"], max_new=s["max_new"],
                                 max_len=s["max_len"], out=s["out"], lse=s["lse"])
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    o, lse = s["out"].clone(), s["lse"].clone()
    if s["seq_start"] is None:  # a token each: all sequences at once
        table = s["table"].long().clamp(0)
        k, v = (x[table].float().transpose(1, 2).reshape(c["n"], hkv, -1, d) for x in (s["k_pages"], s["v_pages"]))
        j = torch.arange(k.shape[2], device="cuda")
        pos = s["length"].long()[:, None] - 1
        seen = j <= pos
        if c["window"]:
            seen &= (j > pos - c["window"]) | (j < c["sinks"])
        v = torch.where((j <= pos)[:, None, :, None], v, 0.0)
        x = torch.matmul(s["q"].float().reshape(c["n"], hkv, -1, d), k.transpose(-1, -2)) / math.sqrt(d)
        x = torch.where(seen[:, None, None], x, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        o[:] = (torch.matmul(p, v) / total).reshape(o.shape).to(o.dtype)
        lse[:] = (top + torch.log(total)).reshape(lse.shape)
        return o, lse
    had, got = _lens(c)  # (a plain program keeps the lengths on the host, too)
    at = 0
    for b, new in enumerate(got):
        n = had[b] + new
        if new == 0:
            continue
        pages = s["table"][b, :-(-n // page)].long()
        pos = torch.arange(n - new, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        seen = j <= pos
        if c["window"]:
            seen &= (j > pos - c["window"]) | (j < c["sinks"])
        k, v = (x[pages].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float() for x in (s["k_pages"], s["v_pages"]))
        q = s["q"][at:at + new].float().reshape(new, hkv, -1, d).permute(1, 2, 0, 3)
        step = max(1, (1 << 30) // (n * new * (hq // hkv)))  # key heads at a time, for the scores' memory
        for h in range(0, hkv, step):
            x = torch.matmul(q[h:h + step], k[h:h + step, None].transpose(-1, -2)) / math.sqrt(d)
            x = torch.where(seen, x, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            total = p.sum(-1, keepdim=True)
            y = torch.matmul(p, v[h:h + step, None]) / total
            heads = slice(h * (hq // hkv), min(hkv, h + step) * (hq // hkv))
            o[at:at + new, heads] = y.permute(2, 0, 1, 3).reshape(new, -1, d).to(o.dtype)
            lse[at:at + new, heads] = (top + torch.log(total))[..., 0].reshape(-1, new).transpose(0, 1)
        at += new
    return o, lse


# --- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    c = case
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "rotate":
        t = c["b"] * c["s"]
        return {"bytes": t * (2.0 * (3 if c["back"] else 2) * (hq + hkv) * d + 4), "flops": t * (hq + hkv) * d * (20.0 if c["back"] else 8.0)}
    had, got = _lens(c)
    t = sum(got)
    if c["op"] == "write":
        return {"bytes": 4.0 * t * (hq + 2 * hkv) * d, "flops": 8.0 * t * (hq + hkv) * d}
    keys = pairs = 0
    for a, new in zip(had, got):
        if new == 0:
            continue
        n = a + new
        if not c["window"]:
            keys += n
            pairs += new * a + new * (new + 1) // 2
            continue
        w, f = c["window"], c["sinks"]
        lo = max(0, a - w + 1)  # the first entry in the first new token's window
        keys += n - lo + min(f, lo)
        # of a token at p: min(p + 1, w) in its window, and min(f, p + 1 - w) first ones before that
        full = max(0, n - max(a, w))  # tokens whose window is full
        part = new - full
        pairs += full * w + part * (a + 1) + part * (part - 1) // 2
        past = range(max(a, w), n)
        ramp = [p for p in past if p + 1 - w < f]
        pairs += sum(p + 1 - w for p in ramp) + f * (len(past) - len(ramp))
    return {"bytes": 4.0 * keys * hkv * d + t * hq * (4.0 * d + 4), "flops": 4.0 * d * hq * pairs}


# --- the same in 64 bits, from the definition ------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "write": _exact_write, "attend": _exact_attend}[case["op"]](s)


def _matrix_rows(c, pos):
    """A turn as complex numbers amp * exp(i * pos * f), [..., 1, R/2]."""
    f = torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(f, c["amp"]).expand(*pos.shape, 1, f.numel()).contiguous(), pos.double()[..., None, None] * f)


def _as_complex(x, c):
    r = c["rot"]
    z = x[..., :r].unflatten(-1, (r // 2, 2)) if c["inter"] else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    return torch.view_as_complex(z.contiguous())


def _from_complex(z, rest, c):
    y = torch.view_as_real(z)
    y = y.flatten(-2) if c["inter"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat([y, rest], -1)


def _exact_turned(x, w, turn, c):
    y = x.double()
    if w is not None:
        y = y / ((y ** 2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    return _from_complex(_as_complex(y, c) * turn, y[..., c["rot"]:], c)


def _exact_rotate(s):
    c = s["case"]
    out = []
    grads = []
    for b in range(c["b"]):  # a batch at a time, for the memory
        turn = _matrix_rows(c, s["pos"][b])
        if not c["back"]:
            out.append([_exact_turned(x[b], w, turn, c).transpose(0, 1) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"]))])
            continue
        row = []
        for dy, x, w in ((s["dq"], s["q"], s["qw"]), (s["dk"], s["k"], s["kw"])):
            dy, x = dy[b].transpose(0, 1).double(), x[b].double()
            g = _from_complex(_as_complex(dy, c) * turn.conj(), dy[..., c["rot"]:], c)
            if w is None:
                row.append((g, None))
                continue
            ms = (x ** 2).mean(-1, keepdim=True) + EPS
            gw = g * w.double()
            # d/dx of x / sqrt(ms): 1 / sqrt(ms) on the diagonal, less x x^T / (D ms^1.5)
            row.append((gw / ms.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (c["d"] * ms ** 1.5), (g * x / ms.sqrt()).sum((0, 1))))
        grads.append(row)
    if not c["back"]:
        return tuple(torch.stack([o[i] for o in out]) for i in range(2))
    dq, dk = (torch.stack([r[i][0] for r in grads]) for i in range(2))
    if not c["norm"]:
        return dq, dk
    return dq, dk, sum(r[0][1] for r in grads), sum(r[1][1] for r in grads)


def _exact_write(s):
    c = s["case"]
    q, k, v = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
    had, got = _lens(c)
    at = 0
    for b, new in enumerate(got):
        if new == 0:
            continue
        slot = torch.arange(had[b], had[b] + new, device="cuda")
        turn = _matrix_rows(c, slot)
        where, row = s["table"][b].long()[slot // c["page"]], slot % c["page"]
        q[at:at + new] = _exact_turned(s["q"][at:at + new], s["qw"], turn, c)
        k[where, :, row] = _exact_turned(s["k"][at:at + new], s["kw"], turn, c)
        v[where, :, row] = s["v"][at:at + new].double()
        at += new
    return q, k, v, None


def _exact_attend(s):
    c = s["case"]
    group, page = c["hq"] // c["hkv"], c["page"]
    o, lse = s["out"].double(), s["lse"].double()
    had, got = _lens(c)
    at = 0
    for b, new in enumerate(got):
        n = had[b] + new
        pages = s["table"][b, :-(-n // page)].long()
        for r in range(0, new, 2048):
            e = min(new, r + 2048)
            first = n - new + r
            # entries that some of these tokens may see
            lo = max(0, first - c["window"] + 1) if c["window"] else 0
            j = torch.cat([torch.arange(0, min(c["sinks"], lo), device="cuda"), torch.arange(lo, n - new + e, device="cuda")])
            p = torch.arange(first, n - new + e, device="cuda")[:, None]
            hide = j > p
            if c["window"]:
                hide |= (j <= p - c["window"]) & (j >= c["sinks"])
            for h in range(c["hkv"]):
                k, v = (x[pages[j // page], h, j % page].double() for x in (s["k_pages"], s["v_pages"]))
                q = s["q"][at + r:at + e, h * group:(h + 1) * group].double()
                x = torch.einsum("igd,jd->gij", q, k) * c["d"] ** -0.5
                x.masked_fill_(hide, -math.inf)
                z = torch.logsumexp(x, -1)
                o[at + r:at + e, h * group:(h + 1) * group] = torch.einsum("gij,jd->igd", torch.exp(x - z[..., None]), v)
                lse[at + r:at + e, h * group:(h + 1) * group] = z.transpose(0, 1)
        at += new
    return o, lse
