"""Cases of the operators around the attention of a decoder layer, and of attention over a shared latent vector a token.

Four operators, in the order in which a serving step calls them:

* ``norm``    residual sum and root-mean-square norm before and after a block: h = residual + scale * gate * u with u the
              block's output or its norm, y = norm of h;
* ``rotate``  rotary positions on query and key heads, with a norm of each head before where the model has one;
* ``store``   a token's latent vector (normed) and its rotary key (rotated) into a paged cache;
* ``latent``  attention of the new tokens over that cache in its absorbed form: a token's key is its latent vector and its
              rotary key, its value the latent vector, for all heads.

Each has a plain form (elementary torch operations in 32 bits, angles in 64), the framework's call, and its definition in
64 bits.  An angle is the position times a pair's frequency; a table holds the frequencies in units of 2^-64 turns.
"""
import math
import random

import torch

own = False

ROPE = 64                                                  # dims of the rotary key beside a latent vector


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm before a block of one decode token: latency, hidden size 5120
        dict(name="norm_t1", op="norm", tokens=1, hidden=5120, post=False, gate=0, wide=False),
        # a verify batch with a norm after the block, a gate for each channel and a residual stream in 32 bits
        dict(name="norm_t61", op="norm", tokens=61, hidden=7168, post=True, gate=1, wide=True),
        # a prompt chunk
        dict(name="norm_t4000", op="norm", tokens=4000, hidden=7168, post=False, gate=0, wide=False),
        # one token of each of 64 requests, halves rotated
        dict(name="rotate_decode_64", op="rotate", tokens=64, heads=64, kv_heads=8, dim=128, part=128, inter=False, normed=False, scaling=0, far=32768),
        # a prompt chunk; heads are normed, half of each is rotated, neighbours pairwise, frequencies of a longer context
        dict(name="rotate_t4000", op="rotate", tokens=4000, heads=40, kv_heads=8, dim=128, part=64, inter=True, normed=True, scaling=2, far=200000),
        # one new token of each of 64 requests
        dict(name="store_decode_64", op="store", tokens=64, latent=512, block=64, inter=True, normed=True, lens=1),
        # a prompt chunk of nine requests
        dict(name="store_t7900", op="store", tokens=7900, latent=512, block=64, inter=True, normed=True, lens=2),
        # a single request's next token after a short prompt: latency
        dict(name="latent_one_1k", op="latent", batch=1, ctx=1000, new=1, block=64, heads=16, latent=512, causal=True, lens=3),
        # ragged decode of 48 requests, small blocks, many heads
        dict(name="latent_decode_48", op="latent", batch=48, ctx=8192, new=1, block=16, heads=96, latent=512, causal=True, lens=4),
        # speculative verification: up to 4 drafted tokens of each of 16 requests
        dict(name="latent_verify_16", op="latent", batch=16, ctx=20000, new=4, block=64, heads=32, latent=512, causal=True, lens=5),
        # a large decode batch with long contexts
        dict(name="latent_decode_long", op="latent", batch=64, ctx=49152, new=1, block=64, heads=64, latent=512, causal=True, lens=6),
        # chunks of prompts over what is cached already, a smaller latent vector
        dict(name="latent_chunk", op="latent", batch=3, ctx=6000, new=300, block=32, heads=20, latent=256, causal=True, lens=7),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "rotate", "store", "latent", "latent", "latent"])
    if op == "norm":
        while True:
            t, h = _log(rng, 1, 8192), 8 * _log(rng, 8, 2048)
            if t * h <= 4000 * 7168:
                return dict(op=op, tokens=t, hidden=h, post=rng.random() < 0.4, gate=rng.choice([0, 0, 1, 2]), wide=rng.random() < 0.3)
    if op == "rotate":
        while True:
            dim = rng.choice([64, 128, 128, 192, 256])
            c = dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.choice([1, 4, 12, 16, 32, 40, 64, 96, 128]), kv_heads=rng.choice([0, 1, 2, 4, 8]), dim=dim,
                     part=rng.choice([dim, dim, dim // 2, 16, 64]), inter=rng.random() < 0.5, normed=rng.random() < 0.4, scaling=rng.randrange(3),
                     far=_log(rng, 100, 1 << 20))
            if c["tokens"] * (c["heads"] + c["kv_heads"]) * dim <= 4000 * 48 * 128:
                return c
    lens, block, latent = rng.randrange(1 << 30), rng.choice([16, 32, 64, 128]), rng.choice([256, 512, 512])
    if op == "store":
        return dict(op=op, tokens=_log(rng, 1, 7900), latent=latent, block=block, inter=rng.random() < 0.5, normed=rng.random() < 0.7, lens=lens)
    while True:
        new = 1 if rng.random() < 0.5 else _log(rng, 1, 16) if rng.random() < 0.7 else _log(rng, 16, 400)
        c = dict(op=op, batch=_log(rng, 1, 128), ctx=_log(rng, 1, 49152), new=new, block=block, heads=rng.choice([1, 4, 8, 12, 16, 20, 32, 40, 64, 96, 128]),
                 latent=latent, causal=rng.random() < 0.85, lens=lens)
        if c["batch"] * c["ctx"] <= 64 * 49152 // 2 and c["batch"] * new * c["heads"] * (c["ctx"] + new) <= 1.2e8:
            return c


def _lens(case):
    """Cached tokens and new tokens of each request: ragged, made from the case alone."""
    r = random.Random(case["lens"])
    if case["op"] == "store":                              # the tokens of up to nine requests, some of them in the middle of a block
        n = min(9, case["tokens"]) if case["tokens"] > 256 else case["tokens"]
        cut = sorted(r.sample(range(1, case["tokens"]), n - 1)) if n > 1 else []
        new = [b - a for a, b in zip([0] + cut, cut + [case["tokens"]])]
        return [r.randrange(4000) for _ in new], new
    ctx = [int(case["ctx"] * (0.25 + 0.75 * r.random())) for _ in range(case["batch"])]
    ctx[r.randrange(len(ctx))] = case["ctx"]
    if case["new"] > 16:
        new = [1 + int((case["new"] - 1) * (0.3 + 0.7 * r.random())) for _ in ctx]
    else:
        new = [1 + r.randrange(case["new"]) for _ in ctx]
    return ctx, new


def work(case):
    op = case["op"]
    if op == "norm":
        t, h = case["tokens"], case["hidden"]
        weights = h * 2 * (1 + case["post"] + (case["gate"] == 1)) + (t * h * 2 if case["gate"] == 2 else 0)
        return dict(bytes=t * h * (4 + (8 if case["wide"] else 4)) + weights, flops=t * h * (6 + 4 * case["post"]))
    if op == "rotate":
        t, rows = case["tokens"], case["tokens"] * (case["heads"] + case["kv_heads"])
        return dict(bytes=4 * rows * case["dim"] + 4 * t + 4 * case["part"], flops=rows * (3 * case["part"] + 4 * case["dim"] * case["normed"]))
    if op == "store":
        t, n = case["tokens"], case["latent"] + ROPE
        return dict(bytes=t * (4 * n + 12) + 2 * case["latent"] * case["normed"], flops=t * (3 * ROPE + 4 * case["latent"] * case["normed"]))
    ctx, new = _lens(case)
    pairs = sum(n * (c + n) - (n * (n - 1) // 2 if case["causal"] else 0) for c, n in zip(ctx, new))
    rows, latent = sum(new) * case["heads"], case["latent"]
    blocks = sum(-(-(c + n) // case["block"]) for c, n in zip(ctx, new))
    return dict(bytes=sum(c + n for c, n in zip(ctx, new)) * (latent + ROPE) * 2 + 4 * blocks + rows * (2 * (latent + ROPE) + 2 * latent + 4),
                flops=2 * pairs * case["heads"] * (2 * latent + ROPE))


# ----------------------------------------------------------------- inputs

def _frequencies(part, scaling):
    """Angles a position of the part/2 pairs, in radians; scaling 1: positions of a context four times as long; 2: only the slow
    pairs' (those that turn fewer than 32 times in 4,096 positions, in full from 1 on)."""
    f = 10000.0 ** (-torch.arange(0, part, 2, dtype=torch.float64) / part)
    if scaling == 1:
        f = f / 4
    if scaling == 2:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / 4 * (1 - keep)
    return f


def _turns(f):
    """Frequencies in units of 2^-64 turns, as the bits of a signed integer."""
    whole = [int(x / (2 * math.pi) * 2.0 ** 64) for x in f.tolist()]
    return torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in whole], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    dev = dict(device="cuda")

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, dtype=torch.float32, device="cuda") * std).to(torch.bfloat16)

    def weight(n):
        return (1 + 0.2 * torch.randn(n, generator=gen, **dev)).to(torch.bfloat16)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, **dev)

    if op == "norm":
        t, h = case["tokens"], case["hidden"]
        x, r = normal(t, h, std=0.7), torch.randn(t, h, generator=gen, **dev) * 3
        x[:, :: 61] *= 12                                  # a few large channels, as activations have
        r[:, 5:: 97] *= 20
        r = r if case["wide"] else r.to(torch.bfloat16)
        return dict(op=op, x=x, residual=r, residual_out=torch.empty_like(r), y=torch.empty_like(x), weight=weight(h), eps=1e-5, scale=0.6 if case["gate"] else 1.0,
                    post=weight(h) if case["post"] else None, gate=None if case["gate"] == 0 else normal(h) if case["gate"] == 1 else normal(t, h))
    if op == "rotate":
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        f = _frequencies(case["part"], case["scaling"])
        qkv = normal(t, hq + 2 * hk, d)
        start = torch.randint(0, case["far"], (), generator=gen, **dev)
        pos = (start + torch.arange(t, **dev)) % case["far"] if t > 256 else torch.randint(0, case["far"], (t,), generator=gen, **dev)
        return dict(op=op, q=qkv[:, :hq], k=qkv[:, hq:hq + hk] if hk else None, positions=pos.to(torch.int32), freq=f.cuda(), turns=_turns(f),
                    amp=0.1 * math.log(4) + 1 if case["scaling"] == 2 else 1.0, inter=case["inter"], offset=d - case["part"],
                    q_norm=weight(d) if case["normed"] else None, k_norm=weight(d) if case["normed"] and hk else None, eps=1e-6,
                    q_out=empty(t, hq, d), k_out=empty(t, hk, d) if hk else None)
    ctx, new = _lens(case)
    total, block, latent = sum(new), case["block"], case["latent"]
    blocks = [-(-(c + n) // block) for c, n in zip(ctx, new)]
    pool = torch.randperm(sum(blocks) + 8, generator=gen, **dev).to(torch.int32)
    nb = torch.tensor(blocks, **dev)
    first, col = torch.cumsum(nb, 0) - nb, torch.arange(max(blocks), **dev)
    table = torch.where(col < nb[:, None], pool[(first[:, None] + col).clamp(max=pool.numel() - 1)], -1).to(torch.int32)
    c, n = torch.tensor(ctx, **dev), torch.tensor(new, **dev)
    offsets = torch.zeros(len(ctx) + 1, dtype=torch.int64, **dev)
    offsets[1:] = torch.cumsum(n, 0)
    req = torch.repeat_interleave(torch.arange(len(ctx), **dev), n)
    pos = c[req] + torch.arange(total, **dev) - offsets[req]
    cache = empty(pool.numel(), block, latent + ROPE)
    for part in cache.view(-1, latent + ROPE).split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=gen, **dev))
    s = dict(op=op, cache=cache, latent=latent, ws=torch.zeros(1 << 27, dtype=torch.uint8, **dev))
    if op == "store":
        f = _frequencies(ROPE, 2)
        both = normal(total, latent + ROPE, std=2.0)       # one projection makes both
        s.update(c=both[:, :latent], k=both[:, latent:], slots=table[req, pos // block].long() * block + pos % block, positions=pos.to(torch.int32),
                 freq=f.cuda(), turns=_turns(f), amp=1.0, inter=case["inter"], norm=weight(latent) if case["normed"] else None, eps=1e-6)
        return s
    q = normal(total, case["heads"], latent + ROPE)
    s.update(q_latent=q[..., :latent], q_rope=q[..., latent:], table=table, q_offsets=offsets.to(torch.int32), kv_lens=(c + n).to(torch.int32),
             softmax_scale=1.5 * (latent + ROPE) ** -0.5, causal=case["causal"], max_kv=max(x + y for x, y in zip(ctx, new)), max_q=max(new),
             out=empty(total, case["heads"], latent), lse=empty(total, case["heads"], dtype=torch.float32))
    return s


# -------------------------------------------------------------------- run

def run(state):
    return _RUN[state["op"]](state)


def _rms(v, w, eps):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * w.float()


def _norm(s):
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        attn.moe_rms_norm(s["x"], s["weight"], s["eps"], s["y"], residual=s["residual"], residual_out=s["residual_out"], scale=s["scale"],
                          gate=s["gate"], post_weight=s["post"])
        return s["y"], s["residual_out"]
    u = s["x"].float()
    if s["post"] is not None:
        u = _rms(u, s["post"], s["eps"])
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["residual"].float() + s["scale"] * u
    return _rms(h, s["weight"], s["eps"]).to(torch.bfloat16), h.to(s["residual"].dtype)


def _turned(x, positions, freq, amp, inter, offset):
    """x [T, heads, dim] in 32 bits with the pairs of dims offset.. rotated."""
    part = 2 * freq.numel()
    angle = positions.double()[:, None] * freq
    cos, sin = (torch.cos(angle) * amp).float()[:, None], (torch.sin(angle) * amp).float()[:, None]
    x = x.clone()
    turn = x[..., offset:offset + part]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if inter else (turn[..., :part // 2], turn[..., part // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    turn.copy_(torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1))
    return x


def _rotate(s):
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        attn.moe_rotary(s["q"], s["positions"], attn.RotaryTable(s["turns"], s["amp"]), s["q_out"], k=s["k"], k_out=s["k_out"],
                        interleaved=s["inter"], offset=s["offset"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"])
        return [v for v in (s["q_out"], s["k_out"]) if v is not None]
    answer = []
    for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])):
        if x is not None:
            x = x.float() if w is None else _rms(x.float(), w, s["eps"])
            answer.append(_turned(x, s["positions"], s["freq"], s["amp"], s["inter"], s["offset"]).to(torch.bfloat16))
    return answer


def _store(s):
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        attn.moe_latent_append(s["c"], s["k"], s["slots"], attn.LatentCache(s["cache"]), s["ws"], positions=s["positions"],
                               table=attn.RotaryTable(s["turns"], s["amp"]), interleaved=s["inter"], norm=s["norm"], eps=s["eps"])
        return s["cache"]
    c = s["c"].float() if s["norm"] is None else _rms(s["c"].float(), s["norm"], s["eps"])
    k = _turned(s["k"].float()[:, None], s["positions"], s["freq"], s["amp"], s["inter"], 0)[:, 0]
    s["cache"].view(-1, s["cache"].shape[2])[s["slots"]] = torch.cat((c, k), 1).to(torch.bfloat16)
    return s["cache"]


def _latent(s):
    if own:
        from block_scaled_fp4_moe_gb300 import attn
        attn.moe_latent_attention(s["q_latent"], s["q_rope"], attn.LatentCache(s["cache"]), s["table"], s["q_offsets"], s["kv_lens"], s["softmax_scale"],
                                  s["out"], s["lse"], s["ws"], causal=s["causal"])
        return s["out"], s["lse"]
    (total, heads, latent), block = s["q_latent"].shape, s["cache"].shape[1]
    batch, max_q = s["table"].shape[0], s["max_q"]
    nb = -(-s["max_kv"] // block)
    keys = s["cache"][s["table"][:, :nb].long().clamp(min=0)].float().view(batch, nb * block, -1)
    lo, kv = s["q_offsets"][:-1].long(), s["kv_lens"].long()
    n = s["q_offsets"][1:].long() - lo
    i, j = torch.arange(max_q, device="cuda"), torch.arange(nb * block, device="cuda")
    rows = (lo[:, None] + i).clamp(max=total - 1)                          # [batch, max_q]
    q = torch.cat((s["q_latent"], s["q_rope"]), -1).float()[rows].view(batch, max_q * heads, -1)
    x = torch.matmul(q, keys.transpose(1, 2)).mul_(s["softmax_scale"]).view(batch, max_q, heads, -1)
    seen = (j < kv[:, None])[:, None, :].expand(batch, max_q, -1)
    if s["causal"]:
        seen = seen & (j <= ((kv - n)[:, None] + i)[..., None])
    x = x.masked_fill_(~seen[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = torch.exp_(x.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, max_q * heads, -1), keys[..., :latent]).view(batch, max_q, heads, latent)
    o = torch.where(l > 0, o / l, 0)
    lse = (m + torch.log(l))[..., 0]
    token = torch.arange(total, device="cuda")
    req = torch.searchsorted(s["q_offsets"].long(), token, right=True) - 1
    return o[req, token - lo[req]].to(torch.bfloat16), lse[req, token - lo[req]]


_RUN = dict(norm=_norm, rotate=_rotate, store=_store, latent=_latent)


# ------------------------------------------------------------------ exact

def _unit(v, eps):
    """Rows of doubles over their root mean square."""
    return v / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + eps)


def _spun(x, s, offset):
    """The rotation as products of complex numbers."""
    part = 2 * s["freq"].numel()
    theta = s["positions"].double()[:, None, None] * s["freq"]
    turn = torch.polar(torch.full_like(theta, s["amp"]), theta)
    old = x[..., offset:offset + part]
    if s["inter"]:
        new = torch.view_as_real(torch.view_as_complex(old.reshape(*old.shape[:-1], part // 2, 2).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(old[..., :part // 2].contiguous(), old[..., part // 2:].contiguous()) * turn
        new = torch.cat((z.real, z.imag), -1)
    return torch.cat((x[..., :offset], new, x[..., offset + part:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        u = s["x"].double()
        if case["post"]:
            u = _unit(u, s["eps"]) * s["post"].double()
        h = s["residual"].double() + s["scale"] * (u if s["gate"] is None else s["gate"].double() * u)
        return _unit(h, s["eps"]) * s["weight"].double(), h
    if op == "rotate":
        answer = []
        for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])):
            if x is not None:
                x = x.double()
                answer.append(_spun(x if w is None else _unit(x, s["eps"]) * w.double(), s, s["offset"]))
        return answer
    latent = s["latent"]
    if op == "store":
        rows = s["cache"].double().view(-1, latent + ROPE)
        c = s["c"].double()
        rows[s["slots"], :latent] = c if s["norm"] is None else _unit(c, s["eps"]) * s["norm"].double()
        rows[s["slots"], latent:] = _spun(s["k"].double()[:, None], s, 0)[:, 0]
        return rows.view(s["cache"].shape)
    total, heads = s["q_latent"].shape[:2]
    out = torch.empty(total, heads, latent, dtype=torch.float64, device="cuda")
    lse = torch.empty(total, heads, dtype=torch.float64, device="cuda")
    ends, kvs, block = s["q_offsets"].tolist(), s["kv_lens"].tolist(), case["block"]
    for b, kv in enumerate(kvs):
        lo, hi = ends[b], ends[b + 1]
        seq = s["cache"][s["table"][b, : -(-kv // block)].long()].double().view(-1, latent + ROPE)[:kv]
        x = torch.einsum("thd,jd->thj", s["q_latent"][lo:hi].double(), seq[:, :latent]) + torch.einsum("thd,jd->thj", s["q_rope"][lo:hi].double(), seq[:, latent:])
        x *= s["softmax_scale"]
        if s["causal"]:
            late = torch.arange(kv, device="cuda")[None] > torch.arange(kv - (hi - lo), kv, device="cuda")[:, None]
            x.masked_fill_(late[:, None], -math.inf)
        lse[lo:hi] = torch.logsumexp(x, -1)
        out[lo:hi] = torch.softmax(x, -1) @ seq[:, :latent]
    return out, lse
