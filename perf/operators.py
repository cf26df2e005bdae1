"""Cases of the prompt and KV-cache operators, for measuring them.

Four operators of serving a language model, in the order a request meets them:

  prompt   attention over whole prompts, packed one behind the other, with
           grouped heads (attention_varlen)
  append   writing K and V into a cache held in 4 bits, and reading the
           entries back (KVCache4.append, KVCache4.read)
  decode   attention of one token per sequence over that cache, with or
           without adding up each entry's attention weight (KVCache4.attend)
  evict    shortening the cache to its entries of highest accumulated weight
           (KVCache4.evict)

The 4-bit format: every 64 channels of a K or V row (one token, one head) hold
a scale s and a minimum m, both bf16, and a code c in 0 .. 15 per value, which
stands for c * s + m.  s = bf16((max - min) / 15), m = bf16(min) and
c = clamp(rint((x - m) / s), 0, 15), or 0 where s is 0.  Value 2i of a row is
the low half of byte i, value 2i + 1 the high half.
"""
import math
import random

import torch

own = False

GROUP = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --- cases -----------------------------------------------------------------------------------------------------------

def listed():
    return [
        # a few chat turns of some tokens each, as a CUDA-graph bucket pads them: launch latency
        dict(name="prompt_short", op="prompt", n=6, longest=61, total=0, pad=9, hq=8, hkv=2, d=64, causal=True, type="fp16", lens=11),
        # four sequences of 1024 tokens with as many key as query heads, attended both ways
        dict(name="prompt_equal", op="prompt", n=4, longest=1024, total=4096, pad=0, hq=16, hkv=16, d=64, causal=False, type="bf16", lens=0),
        # a prefill batch of prompts of many lengths
        dict(name="prompt_packed", op="prompt", n=16, longest=2500, total=0, pad=37, hq=32, hkv=8, d=128, causal=True, type="bf16", lens=12),
        # one long document
        dict(name="prompt_long", op="prompt", n=1, longest=16384, total=16384, pad=0, hq=32, hkv=8, d=128, causal=True, type="bf16", lens=0),
        # the new token of every running sequence
        dict(name="append_token", op="append", n=64, longest=1, total=64, pad=0, hkv=8, d=128, cap=4096, type="bf16", lens=13),
        # a prefill batch's keys and values
        dict(name="append_prompt", op="append", n=12, longest=5000, total=0, pad=21, hkv=8, d=128, cap=8192, type="bf16", lens=14),
        # one user, short history, as many key as query heads: latency
        dict(name="decode_short", op="decode", n=1, longest=701, total=701, hq=16, hkv=16, d=64, cap=1024, weight=False, type="fp16", lens=0),
        # one user, very long history
        dict(name="decode_long", op="decode", n=1, longest=131072, total=131072, hq=32, hkv=8, d=128, cap=131072, weight=False, type="bf16", lens=0),
        # an ordinary batch that keeps eviction weights
        dict(name="decode_batch", op="decode", n=32, longest=4001, total=0, hq=32, hkv=8, d=128, cap=4096, weight=True, type="bf16", lens=15),
        # a full batch of long histories, eight query heads to a key head
        dict(name="decode_full", op="decode", n=64, longest=16000, total=0, hq=64, hkv=8, d=128, cap=16384, weight=True, type="bf16", lens=16),
        # a bounded cache, one entry over its budget after a token: latency
        dict(name="evict_step", op="evict", n=32, longest=2049, total=32 * 2049, hkv=8, d=128, cap=4096, budget=2048, recent=256, lens=0),
        # prompts of up to 8192 tokens cut to a quarter before decoding
        dict(name="evict_prompt", op="evict", n=24, longest=8192, total=0, hkv=8, d=128, cap=8192, budget=2048, recent=512, lens=17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "append", "decode", "evict"])
    d = rng.choice([64, 128])
    kind = rng.choice(["bf16", "fp16"])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    seed = rng.randrange(1, 1 << 30)
    while True:
        n, longest = _log(rng, 1, 64), _log(rng, 1, 16384)
        if op == "prompt":
            c = dict(op=op, n=n, longest=longest, total=0, pad=rng.choice([0, rng.randrange(1, 200)]), hq=0, hkv=rng.choice([1, 2, 4, 8]), d=d,
                     causal=rng.random() < 0.8, type=kind, lens=seed)
            c["hq"] = group * c["hkv"]
            t = sum(_lens(c))
            if t <= 16384 and c["hq"] * t * t <= 32 * 16384 ** 2 and work(c)["flops"] <= work(listed()[3])["flops"]:
                return c
        elif op == "append":
            c = dict(op=op, n=n, longest=_log(rng, 1, 8000), total=0, pad=rng.choice([0, rng.randrange(1, 100)]), hkv=rng.choice([1, 2, 5, 8, 16]), d=d,
                     cap=0, type=kind, lens=seed)
            c["cap"] = c["longest"] + rng.randrange(1, 2000)
            if work(c)["bytes"] <= work(listed()[5])["bytes"] and n * c["cap"] <= 1 << 18:
                return c
        elif op == "decode":
            c = dict(op=op, n=n, longest=_log(rng, 1, 131072), total=0, hq=0, hkv=rng.choice([1, 2, 4, 8]), d=d, cap=0, weight=rng.random() < 0.5,
                     type=kind, lens=seed)
            c["hq"], c["cap"] = group * c["hkv"], c["longest"] + rng.randrange(0, 500)
            if n * c["cap"] * c["hkv"] * d <= 64 * 16384 * 8 * 128 and work(c)["bytes"] <= work(listed()[9])["bytes"]:
                return c
        else:
            c = dict(op=op, n=n, longest=_log(rng, 2, 16384), total=0, hkv=rng.choice([1, 2, 4, 8]), d=d, cap=0, budget=0, recent=0, lens=seed)
            c["cap"] = c["longest"] + rng.randrange(0, 500)
            c["budget"] = rng.randrange(1, c["longest"] + 1)
            c["recent"] = rng.randrange(0, c["budget"] + 1)
            if n * c["cap"] * c["hkv"] * d <= 24 * 8192 * 8 * 128:
                return c


def _lens(c):
    """Lengths of a case's sequences: all equal where it names their total, else spread, the first the longest and some of them empty or of one token."""
    if c["total"]:
        return [c["total"] // c["n"]] * c["n"]
    rng = random.Random(c["lens"])
    got = [c["longest"]]
    for _ in range(c["n"] - 1):
        u = rng.random()
        got.append(0 if u < 0.05 else 1 if u < 0.1 else max(1, int(c["longest"] * rng.uniform(0.05, 1.0))))
    return got


# --- what a program has in hand --------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _starts(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _keys(g, *shape):
    """Rows as keys have them: a few channels carry an offset and a wide spread."""
    x = torch.randn(shape, generator=g, device="cuda")
    wide = torch.ones(shape[-1], device="cuda")
    wide[3::29] = 4.0
    off = torch.zeros(shape[-1], device="cuda")
    off[5::31] = 3.0
    return x * wide + off


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    lens = _lens(c)
    n, hkv, d = c["n"], c["hkv"], c["d"]
    if c["op"] == "prompt":
        rows = sum(lens) + c["pad"]
        # q, k and v are slices of one projection's output
        qkv = torch.randn((rows, c["hq"] + 2 * hkv, d), generator=g, device="cuda").to(TYPES[c["type"]])
        s["q"], s["k"], s["v"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:c["hq"] + hkv], qkv[:, c["hq"] + hkv:]
        s["seq_start"] = _starts(lens)
        s["out"] = torch.zeros((rows, c["hq"], d), dtype=qkv.dtype, device="cuda")
        s["lse"] = torch.zeros((c["hq"], rows), device="cuda")
        return s
    if c["op"] == "append":
        rows = sum(lens) + c["pad"]
        kv = torch.cat([_keys(g, rows, hkv, d), torch.randn((rows, hkv, d), generator=g, device="cuda")], 1).to(TYPES[c["type"]])
        s["k"], s["v"] = kv[:, :hkv], kv[:, hkv:]
        s["seq_start"] = _starts(lens)
        s["length"] = (torch.rand(n, generator=g, device="cuda") * (c["cap"] - torch.tensor(lens, device="cuda") + 1)).int()
        s["length_out"] = torch.zeros_like(s["length"])
        s["k_out"], s["v_out"] = torch.zeros((2, rows, hkv, d), dtype=kv.dtype, device="cuda")
        s["weight"] = torch.rand((n, hkv, c["cap"]), generator=g, device="cuda")
        s["pos"] = torch.full((n, hkv, c["cap"]), -1, dtype=torch.int32, device="cuda")
        k = v = torch.zeros((n, hkv, c["cap"], d), device="cuda", dtype=torch.bfloat16)
    else:
        if c["op"] == "decode":
            k, v = _keys(g, n, hkv, c["cap"], d), torch.randn((n, hkv, c["cap"], d), generator=g, device="cuda")
            s["q"] = torch.randn((n, c["hq"], d), generator=g, device="cuda").to(TYPES[c["type"]])
        else:  # the entries move as they are: any codes do
            k = v = None
        # accumulated weights: a few entries hold most of it, some were never looked at
        w = torch.exp(2.5 * torch.randn((n, hkv, c["cap"]), generator=g, device="cuda") - 4.0)
        s["weight"] = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.05)
        s["length"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # earlier evictions have left the entries in no order
        s["pos"] = torch.argsort(torch.rand(w.shape, generator=g, device="cuda"), -1).int()
        s["weight_out"], s["pos_out"], s["length_out"] = torch.zeros_like(s["weight"]), torch.zeros_like(s["pos"]), torch.zeros_like(s["length"])
    if k is None:
        codes = torch.randint(0, 256, (2, n, hkv, c["cap"], d // 2), generator=g, device="cuda", dtype=torch.uint8)
        meta = torch.randn((2, n, hkv, c["cap"], d // GROUP, 2), generator=g, device="cuda").to(torch.bfloat16)
        s["k_codes"], s["v_codes"], s["k_meta"], s["v_meta"] = codes[0], codes[1], meta[0], meta[1]
    else:
        s["k_codes"], s["k_meta"] = _quantise(k)
        s["v_codes"], s["v_meta"] = _quantise(v)
    if own:  # the framework's handle on these same buffers, which a program makes once
        from io_aware_attention_fwd_gb300 import KVCache4
        s["cache"] = KVCache4(s["k_codes"], s["k_meta"], s["v_codes"], s["v_meta"], s["weight"], s["pos"], s["length"])
    return s


# --- one pass --------------------------------------------------------------------------------------------------------

def run(state):
    return {"prompt": _prompt, "append": _append, "decode": _decode, "evict": _evict}[state["case"]["op"]](state)


def _prompt(s):
    c = s["case"]
    if own:
        from io_aware_attention_fwd_gb300 import attention_varlen
        return attention_varlen(s["q"], s["k"], s["v"], s["seq_start"], causal=c["causal"], out=s["out"], lse=s["lse"])
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    rows, hq, d = q.shape
    hkv = k.shape[1]
    at = torch.arange(rows, device=q.device)
    seq = (at[:, None] >= s["seq_start"][None, 1:]).sum(1)
    seen = seq[:, None] == seq[None, :]
    if c["causal"]:
        seen &= at[None, :] <= at[:, None]
    real = at < s["seq_start"][-1]
    o, lse = s["out"].clone(), s["lse"].clone()
    step = max(1, (1 << 30) // max(1, rows * rows * (hq // hkv)))  # key heads at a time, for the scores' memory
    for h in range(0, hkv, step):
        kk, vv = k[:, h:h + step].transpose(0, 1), v[:, h:h + step].transpose(0, 1)
        e = kk.shape[0]
        qq = q[:, h * (hq // hkv):(h + e) * (hq // hkv)].reshape(rows, e, hq // hkv, d).permute(1, 2, 0, 3)
        x = torch.matmul(qq, kk[:, None].transpose(-1, -2)) / math.sqrt(d)
        x = torch.where(seen, x, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        y = torch.matmul(p, vv[:, None]) / total
        y = y.permute(2, 0, 1, 3).reshape(rows, -1, d).to(o.dtype)
        z = (top + torch.log(total))[..., 0].reshape(-1, rows)
        heads = slice(h * (hq // hkv), (h + e) * (hq // hkv))
        o[:, heads] = torch.where(real[:, None, None], y, o[:, heads])
        lse[heads] = torch.where(real, z, lse[heads])
    return o, lse


def _quantise(x):
    """Codes, packed, and (s, m) of rows of values."""
    x = x.float()
    y = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low, high = y.amin(-1), y.amax(-1)
    m, sc = low.to(torch.bfloat16), ((high - low) / torch.full_like(low, 15.0)).to(torch.bfloat16)  # by a tensor: a true division
    c = torch.round((y - m.float()[..., None]) / sc.float()[..., None]).clamp(0.0, 15.0)
    c = torch.where(sc[..., None] == 0, 0.0, c).to(torch.uint8).reshape(x.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([sc, m], -1)


def _values(codes, meta):
    """The values that codes stand for."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], meta.shape[-2], GROUP).float()
    return (c * meta[..., 0:1].float() + meta[..., 1:2].float()).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _append(s):
    if own:
        cache = s["cache"]
        cache.append(s["k"], s["v"], seq_start=s["seq_start"], length_out=s["length_out"])
        k, v = cache.read(seq_start=s["seq_start"], first_slot=s["length"], k_out=s["k_out"], v_out=s["v_out"])
        return k, v, s["pos"], s["weight"], s["length_out"]
    rows = s["k"].shape[0]
    at = torch.arange(rows, device="cuda")
    seq = (at[:, None] >= s["seq_start"][None, 1:]).sum(1)
    real = (at < s["seq_start"][-1]).nonzero()[:, 0]
    seq = seq[real]
    slot = real - s["seq_start"][seq] + s["length"][seq]
    pos, weight = s["pos"].clone(), s["weight"].clone()
    got = []
    for x, codes, meta, out in ((s["k"], s["k_codes"], s["k_meta"], s["k_out"]), (s["v"], s["v_codes"], s["v_meta"], s["v_out"])):
        c, sm = _quantise(x[real])
        codes[seq, :, slot], meta[seq, :, slot] = c, sm
        y = out.clone()
        y[real] = _values(codes[seq, :, slot], meta[seq, :, slot]).to(y.dtype)
        got.append(y)
    pos[seq, :, slot] = slot.int()[:, None]
    weight[seq, :, slot] = 0.0
    return got[0], got[1], pos, weight, s["length"] + (s["seq_start"][1:] - s["seq_start"][:-1])


def _decode(s):
    c = s["case"]
    if own:
        o, lse = s["cache"].attend(s["q"], weight_out=s["weight_out"] if c["weight"] else None)
        return (o, lse, s["weight_out"]) if c["weight"] else (o, lse)
    k, v = _values(s["k_codes"], s["k_meta"]), _values(s["v_codes"], s["v_meta"])
    n, hkv, cap, d = k.shape
    q = s["q"].float().reshape(n, hkv, -1, d)
    there = (torch.arange(cap, device=q.device)[None] < s["length"][:, None])[:, None]
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    x = torch.where(there[:, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    o = torch.matmul(p, v).reshape(n, -1, d).to(s["q"].dtype)
    lse = (top + torch.log(total)).reshape(n, -1)
    if not c["weight"]:
        return o, lse
    return o, lse, torch.where(there, s["weight"] + p.sum(2), s["weight_out"])


def _evict(s):
    c = s["case"]
    budget, recent = c["budget"], c["recent"]
    if own:
        # the entries move inside the cache's buffers; every move goes from beyond the budget to below it, so calling again moves the same
        s["cache"].evict(budget, recent, weight_out=s["weight_out"], pos_out=s["pos_out"], length_out=s["length_out"])
        return {"k": (s["k_codes"], s["k_meta"]), "v": (s["v_codes"], s["v_meta"]), "weight": s["weight_out"], "pos": s["pos_out"], "length": s["length_out"]}
    n, hkv, cap = s["weight"].shape
    slot = torch.arange(cap, device="cuda")
    held = s["length"].clamp(0, cap)[:, None, None]
    there = slot < held
    newest = torch.where(there, s["pos"], -1).amax(-1, keepdim=True)
    rank = torch.where(s["pos"] > newest - recent, math.inf, s["weight"])
    rank = torch.where(there, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1]
    keep = torch.zeros_like(there.expand(n, hkv, cap)).scatter(-1, order[..., :budget], True) & there
    left = torch.minimum(held, torch.full_like(held, budget))
    # the i-th kept entry beyond the budget goes to the i-th free slot below it
    hole, far = ~keep & (slot < left), keep & (slot >= left)
    from_far = torch.sort(torch.where(far, slot, cap), -1)[0]
    nth = (hole.long().cumsum(-1) - 1).clamp(0)
    src = torch.where(hole, torch.gather(from_far, -1, nth), slot)
    src = torch.where(slot < left, src, slot)
    out = {}
    for name in ("k", "v"):
        out[name] = tuple(torch.gather(x.reshape(n, hkv, cap, -1), 2, src[..., None].expand(-1, -1, -1, x[0, 0, 0].numel())).reshape(x.shape)
                          for x in (s[name + "_codes"], s[name + "_meta"]))
    out["weight"] = torch.where(slot < left, torch.gather(s["weight"], -1, src), s["weight_out"])
    out["pos"] = torch.where(slot < left, torch.gather(s["pos"], -1, src), s["pos_out"])
    out["length"] = left[:, 0, 0].int()
    return out


# --- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    c, lens = case, _lens(case)
    d, hkv, t = c["d"], c["hkv"], sum(_lens(case))
    entry = 2 * (d // 2 + 4 * (d // GROUP))  # K and V of one token and head, in 4 bits
    if c["op"] == "prompt":
        pairs = sum(x * (x + 1) // 2 if c["causal"] else x * x for x in lens)
        return {"bytes": 4.0 * t * (c["hq"] + hkv) * d + 4.0 * t * c["hq"], "flops": 4.0 * d * c["hq"] * pairs}
    if c["op"] == "append":  # K and V in, written, read back and out; a position and a weight to an entry
        return {"bytes": t * hkv * (8.0 * d + 2 * entry + 8), "flops": 16.0 * t * hkv * d}
    if c["op"] == "decode":
        return {"bytes": t * hkv * (entry + (8.0 if c["weight"] else 0.0)) + c["n"] * c["hq"] * (4.0 * d + 4), "flops": 4.0 * d * c["hq"] * t}
    total = 0.0
    for x in lens:
        left = min(x, c["budget"])
        free = max(0, x - left)
        moved = free * (left / x) if x else 0.0  # of `left` kept entries, the share that lies beyond the budget
        total += hkv * (8.0 * x + 8.0 * left + 2 * entry * moved)
    return {"bytes": total, "flops": 4.0 * hkv * t}


# --- the same in 64 bits, from the definition ------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "append": _exact_append, "decode": _exact_decode, "evict": _exact_evict}[case["op"]](s)


def _exact_prompt(s):
    c = s["case"]
    o, lse = s["out"].double(), s["lse"].double()
    at = s["seq_start"].tolist()
    group = c["hq"] // c["hkv"]
    for a, b in zip(at, at[1:]):
        if a == b:
            continue
        for h in range(c["hq"]):
            q, k, v = s["q"][a:b, h].double(), s["k"][a:b, h // group].double(), s["v"][a:b, h // group].double()
            for r in range(0, b - a, 4096):
                e = min(b - a, r + 4096)
                n = e if c["causal"] else b - a
                x = q[r:e] @ k[:n].T * c["d"] ** -0.5
                if c["causal"]:
                    x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu(r + 1), -math.inf)
                z = torch.logsumexp(x, 1)
                o[a + r:a + e, h] = torch.exp(x - z[:, None]) @ v[:n]
                lse[h, a + r:a + e] = z
    return o, lse


def _exact_rows(x):
    """Values of rows after the 4-bit format, from 64-bit arithmetic on its definition."""
    y = x.double().unflatten(-1, (-1, GROUP))
    low = y.min(-1, keepdim=True).values
    m = low.bfloat16().double()
    sc = ((y.max(-1, keepdim=True).values - low) / 15).bfloat16().double()
    code = ((y - m) / sc.where(sc != 0, torch.ones_like(sc))).round().clamp(0, 15)
    return (code * sc + m).flatten(-2)


def _exact_append(s):
    k, v = s["k_out"].double(), s["v_out"].double()
    t = int(s["seq_start"][-1])
    k[:t], v[:t] = _exact_rows(s["k"][:t]), _exact_rows(s["v"][:t])
    weight = s["weight"].double()
    at = s["seq_start"].tolist()
    for b, n in enumerate(s["length"].tolist()):
        weight[b, :, n:n + at[b + 1] - at[b]] = 0
    return k, v, None, weight, None


def _exact_decode(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    o = torch.zeros((c["n"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["n"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    weight = s["weight_out"].double()
    shift = torch.tensor([0, 4], device="cuda", dtype=torch.uint8)
    for b, n in enumerate(s["length"].tolist()):
        if n == 0:
            continue
        rows = []
        for name in ("k", "v"):
            code = (s[name + "_codes"][b, :, :n, :, None] >> shift) & 15
            sm = s[name + "_meta"][b, :, :n].double().repeat_interleave(GROUP, dim=2)
            rows.append(code.flatten(-2).double() * sm[..., 0] + sm[..., 1])
        q = s["q"][b].double().unflatten(0, (c["hkv"], group))
        x = torch.einsum("hgd,hjd->hgj", q, rows[0]) * c["d"] ** -0.5
        p = torch.softmax(x, -1)
        o[b] = torch.einsum("hgj,hjd->hgd", p, rows[1]).flatten(0, 1)
        lse[b] = torch.logsumexp(x, -1).flatten()
        weight[b, :, :n] = s["weight"][b, :, :n].double() + p.sum(1)
    return (o, lse, weight) if c["weight"] else (o, lse)


def _exact_evict(s):
    """Entry by entry on the host, from the definition."""
    c = s["case"]
    budget, recent = c["budget"], c["recent"]
    meta = {name: s[name + "_meta"].double().cpu() for name in ("k", "v")}
    w, p, n = s["weight"].double().cpu(), s["pos"].cpu(), s["length"].tolist()
    out_w = s["weight_out"].double().cpu()
    for b in range(c["n"]):
        left = min(n[b], budget)
        for h in range(c["hkv"]):
            weight, pos = w[b, h, :n[b]].tolist(), p[b, h, :n[b]].tolist()
            newest = max(pos, default=0)
            order = sorted(range(n[b]), key=lambda j: (pos[j] <= newest - recent, -weight[j] if pos[j] <= newest - recent else 0.0, j))
            kept = set(order[:left])
            src = list(range(left))
            holes = [j for j in range(left) if j not in kept]
            for hole, far in zip(holes, sorted(j for j in kept if j >= left)):
                src[hole] = far
            if left:
                out_w[b, h, :left] = w[b, h, src]
                for m in meta.values():
                    m[b, h, :left] = m[b, h, src]
    return {"k": [None, meta["k"].cuda()], "v": [None, meta["v"].cuda()], "weight": out_w.cuda(), "pos": None, "length": None}
