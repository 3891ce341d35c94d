"""Cases of the attention half of a decoder layer in 8 bits: what runs between two MoE layers of a decode step.

Four operators, in the order in which a serving step calls them:

* ``tables``     block tables and slot maps from the requests' lengths;
* ``project``    y = x W^T with E4M3 operands and a power-of-two scale for each block of 128;
* ``append``     new keys and values into the paged E4M3 cache, one scale for each block of tokens and head;
* ``attend``     attention of the new tokens over that cache.

Each has a plain form (elementary torch operations in 32 bits), the framework's call, and its definition in 64 bits.
Shared definition of the 8-bit formats: a group of values with largest finite magnitude a is stored as E4M3 codes
(nearest even) of v / 2^e, where e is the smallest exponent with a <= 448 * 2^e, at least -126; the scale is the
byte e + 127.  Values that are not finite become the NaN code.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 running requests
        dict(name="tables_decode_64", op="tables", batch=64, ctx=8192, new=1, block=64, lens=1),
        # a mixed step: 1,000 requests, most decoding, some with a chunk of their prompt, small blocks
        dict(name="tables_mixed_1000", op="tables", batch=1000, ctx=4096, new=96, block=16, lens=2),
        # the attention input projection (query, key and value heads) of a single token: hidden size 5120
        dict(name="project_t1", op="project", tokens=1, n=7168, k=5120),
        # a verify batch through the attention output projection, hidden size 7168, an odd token count
        dict(name="project_t61", op="project", tokens=61, n=7168, k=8192),
        # a prompt chunk through the input projection
        dict(name="project_t4000", op="project", tokens=4000, n=7168, k=5120),
        # one new token of each of 64 requests
        dict(name="append_decode_64", op="append", batch=64, ctx=8000, new=1, block=64, kv_heads=8, group=8, dim=128, lens=3),
        # a chunk of 4,000 and some prompt tokens of nine requests
        dict(name="append_prompt", op="append", batch=9, ctx=3000, new=880, block=64, kv_heads=8, group=5, dim=128, lens=4),
        # a single request's next token after a short prompt: latency
        dict(name="attend_one_1k", op="attend", batch=1, ctx=1000, new=1, block=64, kv_heads=8, group=5, dim=128, causal=True, window=0, lens=5),
        # ragged decode of 48 requests, small blocks
        dict(name="attend_decode_48", op="attend", batch=48, ctx=8192, new=1, block=16, kv_heads=8, group=8, dim=128, causal=True, window=0, lens=6),
        # speculative verification: up to 4 drafted tokens of each of 16 requests
        dict(name="attend_verify_16", op="attend", batch=16, ctx=20000, new=4, block=64, kv_heads=8, group=12, dim=128, causal=True, window=0, lens=7),
        # a large decode batch with long contexts
        dict(name="attend_decode_long", op="attend", batch=64, ctx=49152, new=1, block=64, kv_heads=8, group=8, dim=128, causal=True, window=0, lens=8),
        # chunks of prompts over what is cached already, head size 64
        dict(name="attend_chunk", op="attend", batch=3, ctx=9000, new=500, block=32, kv_heads=8, group=6, dim=64, causal=True, window=0, lens=9),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "project", "append", "attend", "attend"])
    lens = rng.randrange(1 << 30)
    if op == "tables":
        return dict(op=op, batch=_log(rng, 1, 2000), ctx=_log(rng, 1, 16384), new=_log(rng, 1, 64), block=rng.choice([16, 32, 64, 128]), lens=lens)
    if op == "project":
        while True:
            t, n, k = _log(rng, 1, 4000), _log(rng, 64, 16384), 16 * _log(rng, 8, 1024)
            if t * n * k <= 4000 * 7168 * 5120:
                return dict(op=op, tokens=t, n=n, k=k)
    heads = dict(block=rng.choice([16, 32, 64, 128]), kv_heads=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16]),
                 dim=rng.choice([64, 128, 128]), lens=lens)
    if op == "append":
        while True:
            c = dict(op=op, batch=_log(rng, 1, 256), ctx=_log(rng, 1, 8192), new=_log(rng, 1, 1000), **heads)
            if c["batch"] * c["new"] <= 8192 and c["batch"] * c["ctx"] <= 1 << 19:
                return c
    while True:
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 16) if rng.random() < 0.7 else _log(rng, 16, 600)
        c = dict(op=op, batch=_log(rng, 1, 128), ctx=_log(rng, 1, 49152), new=new, **heads, causal=rng.random() < 0.8,
                 window=_log(rng, 16, 8192) if rng.random() < 0.25 else 0)
        pairs = c["batch"] * new * c["kv_heads"] * c["group"] * (c["ctx"] + new)
        if c["batch"] * c["ctx"] * c["kv_heads"] * c["dim"] <= 64 * 49152 * 8 * 128 // 2 and pairs <= 1.7e8:
            return c


def _lens(case):
    """Cached tokens and new tokens of each request: ragged, made from the case alone."""
    r = random.Random(case["lens"])
    ctx = [int(case["ctx"] * (0.25 + 0.75 * r.random())) for _ in range(case["batch"])]
    ctx[r.randrange(len(ctx))] = case["ctx"]
    if case["op"] == "tables" and case["new"] > 1:       # most requests decode, some bring a chunk of their prompt
        new = [1 if r.random() < 0.9 else 1 + r.randrange(case["new"]) for _ in ctx]
    elif case["new"] > 16:
        new = [1 + int(case["new"] * (0.3 + 0.7 * r.random())) for _ in ctx]
    else:
        new = [1 + r.randrange(case["new"]) for _ in ctx]
    if case["op"] != "attend" and len(ctx) > 2:          # a request that joins: nothing cached
        ctx[0] = 0
    return ctx, new


def _blocks(ctx, new, block):
    """Blocks that a request holds before and after the step, and its width in the table."""
    before = [-(-c // block) for c in ctx]
    after = [-(-(c + n) // block) for c, n in zip(ctx, new)]
    return before, after, max(after)


def work(case):
    op = case["op"]
    if op == "project":
        t, n, k = case["tokens"], case["n"], case["k"]
        return dict(bytes=t * k * 2 + n * k + (-(-n // 128)) * (-(-k // 128)) + t * n * 2, flops=2 * t * n * k)
    ctx, new = _lens(case)
    total = sum(new)
    before, after, _ = _blocks(ctx, new, case["block"])
    if op == "tables":
        made = sum(after) - sum(before)
        return dict(bytes=8 * len(ctx) + 8 * made + 8 * len(ctx) + 12 * total + 8, flops=0)
    hkv, d, block = case["kv_heads"], case["dim"], case["block"]
    if op == "append":
        # new values in, codes and scales out, the slot map; the held codes of a block need a pass only where its scale grows
        touched = sum(-(-(c + n) // block) - c // block for c, n in zip(ctx, new))
        return dict(bytes=total * (hkv * d * 2 * (2 + 1) + 8) + touched * hkv * 2, flops=0)
    read = pairs = 0
    for c, n in zip(ctx, new):
        kv, w = c + n, case["window"]
        for i in range(n):
            hi = c + i + 1 if case["causal"] else kv
            pairs += hi - (max(0, c + i + 1 - w) if w else 0)
        read += kv - (max(0, c + 1 - w) if w else 0)
    heads = hkv * case["group"]
    return dict(bytes=read * hkv * d * 2 + sum(after) * (4 + 2 * hkv) + total * heads * (4 * d + 4), flops=4 * pairs * heads * d)


# ----------------------------------------------------------------- inputs

def _table(ctx, new, block, gen):
    """A pool of blocks in random order, given out to the requests: (table of the held blocks, all blocks, pool)."""
    before, after, width = _blocks(ctx, new, block)
    pool = torch.randperm(sum(after) + 8, generator=gen, device="cuda").to(torch.int32)
    b = torch.tensor(before, device="cuda")
    first = torch.cumsum(b, 0) - b
    col = torch.arange(width, device="cuda")
    at = first[:, None] + col
    held = torch.where(col < b[:, None], pool[at.clamp(max=pool.numel() - 1)], -1).to(torch.int32)
    return held, pool[sum(before):].clone(), pool.numel()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    dev = dict(device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float32, device="cuda").to(torch.bfloat16)

    if op == "project":
        t, n, k = case["tokens"], case["n"], case["k"]
        x = normal(t, k)
        x[:, :: 61] *= 12                                # a few large channels, as activations have
        w = (torch.randn(n, k, generator=gen, **dev) * 120).clamp(-448, 448).to(E4M3)
        scale = torch.randint(112, 117, (-(-n // 128), -(-k // 128)), generator=gen, dtype=torch.uint8, **dev)
        return dict(op=op, x=x, w=w.view(torch.uint8), scale=scale, y=torch.empty(t, n, dtype=torch.bfloat16, **dev),
                    ws=torch.zeros((1 << 22) + 2 * t * k, dtype=torch.uint8, **dev))
    ctx, new = _lens(case)
    total, block = sum(new), case["block"]
    held, free, nblocks = _table(ctx, new, block, gen)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(op=op, block=block, total=total, ctx=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), table=held,
             ws=torch.zeros(1 << 26, dtype=torch.uint8, **dev))
    if op == "tables":
        batch = len(ctx)
        s.update(free=free, head=torch.zeros(1, **i32), head_out=torch.empty(1, **i32), kv_lens=torch.empty(batch, **i32),
                 q_offsets=torch.empty(batch + 1, **i32), slots=torch.empty(total, dtype=torch.int64, **dev), positions=torch.empty(total, **i32))
        return s
    hkv, group, d = case["kv_heads"], case["group"], case["dim"]
    # the whole table, and where every new token goes
    c, n = s["ctx"].long(), s["new"].long()
    b, a = -(-c // block), -(-(c + n) // block)
    col = torch.arange(held.shape[1], device="cuda")
    grown = (col >= b[:, None]) & (col < a[:, None])
    held[grown] = free[: int(grown.sum())]
    req = torch.repeat_interleave(torch.arange(len(ctx), device="cuda"), n)
    offsets = torch.zeros(len(ctx) + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(n, 0)
    pos = c[req] + torch.arange(total, device="cuda") - offsets[req]
    s["slots"] = held[req, pos // block].long() * block + pos % block
    # codes of values with a standard deviation near 1, each block and head with a size of its own
    shape = (nblocks, hkv, block // 16, 16 * d)
    codes = []
    for _ in range(2):
        u = torch.empty(shape, dtype=torch.uint8, **dev)
        for part in u.split(max(1, (1 << 28) // (hkv * block * d))):
            part.copy_((torch.randn(part.shape, generator=gen, **dev) * 100).clamp_(-448, 448).to(E4M3).view(torch.uint8))
        codes.append(u)
    s["k_cache"] = codes[0].view(nblocks, hkv, block // 16, d // 16, 16, 16)
    s["v_cache"] = codes[1].view(nblocks, hkv, block // 16, d, 16)
    s["k_scale"], s["v_scale"] = (torch.randint(119, 122, (nblocks, hkv), generator=gen, dtype=torch.uint8, **dev) for _ in range(2))
    qkv = normal(total, (group + 2) * hkv, d)
    if op == "append":
        qkv *= torch.exp2(torch.randint(-2, 3, (total, 1, 1), generator=gen, **dev)).to(torch.bfloat16)
        s.update(k=qkv[:, group * hkv:(group + 1) * hkv], v=qkv[:, (group + 1) * hkv:])
        return s
    s.update(q=qkv[:, : group * hkv], kv_lens=(c + n).to(torch.int32), q_offsets=offsets.to(torch.int32), softmax_scale=d ** -0.5,
             causal=case["causal"], window=case["window"], max_kv=max(x + y for x, y in zip(ctx, new)), max_q=max(new),
             out=torch.empty(total, group * hkv, d, dtype=torch.bfloat16, **dev), lse=torch.empty(total, group * hkv, dtype=torch.float32, **dev))
    return s


# -------------------------------------------------------------------- run

def run(state):
    return _RUN[state["op"]](state)


def _tables(s):
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        attn.moe_kv_build_tables(s["ctx"], s["new"], s["block"], s["free"], s["head"], s["table"], s["kv_lens"], s["q_offsets"], s["slots"],
                                 s["positions"], s["head_out"], s["ws"])
        return s["table"], s["kv_lens"], s["q_offsets"], s["slots"], s["positions"], s["head_out"]
    c, n, block = s["ctx"].long(), s["new"].long(), s["block"]
    kv = c + n
    before, after = (c + block - 1) // block, (kv + block - 1) // block
    made = after - before
    first = s["head"].long() + torch.cumsum(made, 0) - made
    col = torch.arange(s["table"].shape[1], device="cuda")
    grown = (col >= before[:, None]) & (col < after[:, None])
    at = first[:, None] + col - before[:, None]
    table = torch.where(grown, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"])
    offsets = torch.zeros(n.numel() + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(n, 0)
    token = torch.arange(s["total"], device="cuda")
    req = torch.searchsorted(offsets, token, right=True) - 1
    pos = c[req] + token - offsets[req]
    slots = table[req, pos // block].long() * block + pos % block
    head = s["head"] + made.sum().to(torch.int32)
    return table, kv.to(torch.int32), offsets.to(torch.int32), slots, pos.to(torch.int32), head


def _exponent(a):
    """The smallest e >= -126 with a <= 448 * 2^e, elementwise."""
    m, e = torch.frexp(a)
    return (e - 9 + (m > 0.875)).clamp(min=-126)


def _codes(v, e):
    """E4M3 values of v / 2^e, held in 8 bits."""
    q = torch.ldexp(v, -e)
    return torch.where(torch.isfinite(v), q, math.nan).to(E4M3)


def _amax(v, dim):
    return torch.where(torch.isfinite(v), v.abs(), 0).amax(dim)


def _project(s):
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        attn.moe_linear_fp8(s["x"], attn.FP8Weight(s["w"], s["scale"]), s["y"], s["ws"])
        return s["y"]
    t, k = s["x"].shape
    kb = s["scale"].shape[1]
    x = torch.nn.functional.pad(s["x"].float(), (0, kb * 128 - k)).view(t, kb, 128)
    e = _exponent(_amax(x, 2))[..., None]
    x = torch.ldexp(_codes(x, e).float(), e).view(t, kb * 128)[:, :k]
    scale = torch.ldexp(torch.ones((), device="cuda"), s["scale"].int() - 127)
    scale = scale.repeat_interleave(128, 0)[: s["w"].shape[0]].repeat_interleave(128, 1)[:, :k]
    return torch.matmul(x, (s["w"].view(E4M3).float() * scale).t()).to(torch.bfloat16)


def _append(s):
    kc, vc, ks, vs = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        attn.moe_kv_append(s["k"], s["v"], s["slots"], attn.KVCache(kc, vc, ks, vs), s["ws"])
        return kc.view(E4M3), vc.view(E4M3), ks, vs
    block, (t, hkv, d) = s["block"], s["k"].shape
    blk, off = s["slots"] // block, s["slots"] % block
    lead = torch.ones_like(blk, dtype=torch.bool)
    lead[1:] = blk[1:] != blk[:-1]
    of = torch.cumsum(lead, 0) - 1                       # the run of tokens in one block that a token is of
    at, start = blk[lead], off[lead]
    index = torch.arange(block, device="cuda").view(-1, 16)
    for cache, scale, x, old in ((kc, ks, s["k"].float(), (index < start[:, None, None])[:, None, :, None, :, None]),
                                 (vc, vs, s["v"].float(), (index < start[:, None, None])[:, None, :, None, :])):
        a = torch.zeros(at.numel(), hkv, device="cuda").index_reduce_(0, of, _amax(x, 2), "amax")
        e = _exponent(a)
        was = scale[at].int() - 127
        e = torch.where(start[:, None] > 0, torch.maximum(e, was), e)
        held = cache[at]
        shape = (-1, hkv) + (1,) * (held.dim() - 2)
        again = _codes(held.view(E4M3).float(), (e - was).view(shape)).view(torch.uint8)
        cache[at] = torch.where(old & (e > was).view(shape), again, held)
        scale[at] = (e + 127).to(torch.uint8)
        codes = _codes(x, e[of][..., None]).view(torch.uint8)
        if cache is kc:
            cache[blk, :, off // 16, :, off % 16, :] = codes.view(t, hkv, d // 16, 16)
        else:
            cache[blk, :, off // 16, :, off % 16] = codes
    return kc.view(E4M3), vc.view(E4M3), ks, vs


def _attend(s):
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        cache = attn.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        attn.moe_kv_attention(s["q"], cache, s["table"], s["q_offsets"], s["kv_lens"], s["softmax_scale"], s["out"], s["lse"], s["ws"],
                              causal=s["causal"], window=s["window"])
        return s["out"], s["lse"]
    (total, heads, d), hkv, block = s["q"].shape, s["k_cache"].shape[1], s["block"]
    group, batch, max_q = heads // hkv, s["table"].shape[0], s["max_q"]
    nb = -(-s["max_kv"] // block)
    pages = s["table"][:, :nb].long().clamp(min=0)
    k = s["k_cache"][pages].view(E4M3).float()
    k = k * torch.ldexp(torch.ones((), device="cuda"), s["k_scale"][pages].int() - 127)[..., None, None, None, None]
    k = k.permute(0, 2, 1, 3, 5, 4, 6).reshape(batch, hkv, nb * block, d)
    v = s["v_cache"][pages].view(E4M3).float()
    v = v * torch.ldexp(torch.ones((), device="cuda"), s["v_scale"][pages].int() - 127)[..., None, None, None]
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(batch, hkv, nb * block, d)
    lo, kv = s["q_offsets"][:-1].long(), s["kv_lens"].long()
    n = s["q_offsets"][1:].long() - lo
    i = torch.arange(max_q, device="cuda")
    rows = (lo[:, None] + i).clamp(max=total - 1)                          # [batch, max_q]
    q = s["q"].float()[rows].view(batch, max_q, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, max_q * group, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["softmax_scale"]).view(batch, hkv, max_q, group, nb * block)
    j = torch.arange(nb * block, device="cuda")
    pos = (kv - n)[:, None] + i
    seen = (j < kv[:, None])[:, None, :].expand(batch, max_q, -1)
    if s["causal"]:
        seen = seen & (j <= pos[..., None])
    if s["window"]:
        seen = seen & (j > pos[..., None] - s["window"])
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = torch.exp_(x.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, hkv, max_q * group, -1), torch.where((j < kv[:, None])[:, None, :, None], v, 0)).view(batch, hkv, max_q, group, d)
    o = torch.where(l > 0, o / l, 0)
    lse = (m + torch.log(l))[..., 0]
    token = torch.arange(total, device="cuda")
    req = torch.searchsorted(s["q_offsets"].long(), token, right=True) - 1
    at = token - lo[req]
    return (o[req, :, at].reshape(total, heads, d).to(torch.bfloat16), lse[req, :, at].reshape(total, heads))


_RUN = dict(tables=_tables, project=_project, append=_append, attend=_attend)


# ------------------------------------------------------------------ exact

def _e4m3_of(v):
    """The nearest E4M3 number of each double of magnitude at most 448, ties to the even code."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _least(a):
    """2^e of the shared definition, from doubles."""
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448) - 1e-9).clamp(min=-126)
    e = torch.where(a > 448 * torch.exp2(e), e + 1, e)
    return torch.exp2(torch.where((a <= 448 * torch.exp2(e - 1)) & (e > -126), e - 1, e))


def _value(code):
    """The numbers of E4M3 codes (finite ones), from their bits."""
    c = code.to(torch.int64)
    ex, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex == 0, man * 2.0 ** -9, (8 + man) * torch.exp2(ex.double() - 10))
    return torch.where(c >= 128, -mag, mag)


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None                                       # whole numbers
    s = prepare(case, seed)
    if op == "project":
        x, w = s["x"].double(), _value(s["w"])
        for b in range(s["scale"].shape[1]):
            cols = slice(128 * b, min(128 * (b + 1), x.shape[1]))
            unit = _least(x[:, cols].abs().amax(1, keepdim=True))
            x[:, cols] = _e4m3_of(x[:, cols] / unit) * unit
            w[:, cols] *= torch.exp2(s["scale"][torch.arange(w.shape[0], device="cuda") // 128, b].double() - 127)[:, None]
        return x @ w.t()
    if op == "append":
        t, hkv, d = s["k"].shape
        block, slots = s["block"], s["slots"].tolist()
        answer = []
        for cache, scale, x, is_k in ((s["k_cache"], s["k_scale"], s["k"].double(), True), (s["v_cache"], s["v_scale"], s["v"].double(), False)):
            nb = cache.shape[0]
            c = _value(cache)                             # as [block, head, token, dim]
            c = c.permute(0, 1, 2, 4, 3, 5).reshape(nb, hkv, block, d) if is_k else c.permute(0, 1, 2, 4, 3).reshape(nb, hkv, block, d)
            i = 0
            while i < t:
                n = i + 1
                while n < t and slots[n] // block == slots[i] // block:
                    n += 1
                b, o = divmod(slots[i], block)
                unit = _least(x[i:n].abs().amax((0, 2)))
                if o:
                    was = torch.exp2(scale[b].double() - 127)
                    unit = torch.maximum(unit, was)
                    c[b, :, :o] = _e4m3_of(c[b, :, :o] * (was / unit)[:, None, None])
                c[b, :, o:o + n - i] = _e4m3_of(x[i:n] / unit[:, None]).permute(1, 0, 2)
                i = n
            if is_k:
                answer.append(c.view(nb, hkv, block // 16, 16, d // 16, 16).permute(0, 1, 2, 4, 3, 5).contiguous())
            else:
                answer.append(c.view(nb, hkv, block // 16, 16, d).permute(0, 1, 2, 4, 3).contiguous())
        return answer[0], answer[1], None, None
    total, heads, d = s["q"].shape
    hkv, block = s["k_cache"].shape[1], s["block"]
    group = heads // hkv
    out = torch.empty(total, heads, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(total, heads, dtype=torch.float64, device="cuda")
    ends, kvs = s["q_offsets"].tolist(), s["kv_lens"].tolist()
    for b, kv in enumerate(kvs):
        lo, hi = ends[b], ends[b + 1]
        page = s["table"][b, : -(-kv // block)].long()
        for h in range(hkv):
            k = _value(s["k_cache"][page, h]) * torch.exp2(s["k_scale"][page, h].double() - 127)[:, None, None, None, None]
            v = _value(s["v_cache"][page, h]) * torch.exp2(s["v_scale"][page, h].double() - 127)[:, None, None, None]
            k = k.transpose(2, 3).reshape(-1, d)[:kv]
            v = v.transpose(2, 3).reshape(-1, d)[:kv]
            q = s["q"][lo:hi, h * group:(h + 1) * group].double()
            x = torch.einsum("ngd,jd->ngj", q, k) * s["softmax_scale"]
            at = torch.arange(kv - (hi - lo), kv, device="cuda")[:, None]
            j = torch.arange(kv, device="cuda")[None]
            hide = torch.zeros(hi - lo, kv, dtype=torch.bool, device="cuda")
            if s["causal"]:
                hide |= j > at
            if s["window"]:
                hide |= j <= at - s["window"]
            x[hide[:, None].expand_as(x)] = -math.inf
            lse[lo:hi, h * group:(h + 1) * group] = torch.logsumexp(x, -1)
            out[lo:hi, h * group:(h + 1) * group] = torch.softmax(x, -1).nan_to_num(0.0) @ v
    return out, lse
