"""The attention half on the GPU against its definitions in 64 bits
(attn_reference): tables and cache contents exactly, attention and projection
within bounds derived from the kernels' arithmetic (stated in the reference)."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attn_reference as ref
from block_scaled_fp4_moe_gb300 import _build, attn, moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def workspace(n=1 << 25):
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    return ws


def status(ws):
    return moe.moe_check_device_status(ws)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def bf16(a):
    return torch.tensor(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


class Guarded:
    """A tensor inside a larger buffer whose margins must keep their bytes."""

    def __init__(self, shape, dtype, fill=0xA5, margin=4096):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.buf = torch.full((2 * margin + n,), fill, dtype=torch.uint8, device="cuda")
        self.t = self.buf[margin:margin + n].view(dtype).view(shape)
        self.margin, self.fill, self.n = margin, fill, n

    def check(self):
        b = self.buf.cpu().numpy()
        assert (b[: self.margin] == self.fill).all() and (b[self.margin + self.n:] == self.fill).all()


# ------------------------------------------------------------------ tables

def run_tables(ctx, new, size, free, head, table, t_max, ws):
    B = len(ctx)
    g = dict(table=Guarded(table.shape, torch.int32), kv=Guarded((B,), torch.int32), qo=Guarded((B + 1,), torch.int32),
             slots=Guarded((t_max,), torch.int64), pos=Guarded((t_max,), torch.int32), head=Guarded((1,), torch.int32))
    g["table"].t.copy_(i32(table))
    before = {k: v.buf.clone() for k, v in g.items()}
    attn.moe_kv_build_tables(i32(ctx), i32(new), size, i32(free), i32([head]), g["table"].t, g["kv"].t, g["qo"].t, g["slots"].t,
                             g["pos"].t, g["head"].t, ws)
    st = status(ws)
    for v in g.values():
        v.check()
    return st, {k: v.t.cpu().numpy() for k, v in g.items()}, all(torch.equal(before[k], g[k].buf) for k in g)


@pytest.mark.parametrize("B,size,ctx_max,new_max,spare", [
    (1, 16, 0, 1, 0), (1, 128, 5, 700, 3), (3, 16, 100, 1, 0), (64, 64, 5000, 1, 9), (65, 32, 300, 40, 0), (513, 16, 64, 9, 100),
    (1500, 64, 900, 2, 0), (8192, 16, 40, 2, 5)])
def test_tables_match_the_definition(B, size, ctx_max, new_max, spare):
    rng = np.random.default_rng(B + size)
    ctx = rng.integers(0, ctx_max + 1, B)
    new = rng.integers(0, new_max + 1, B)                  # requests without a new token among them
    ctx[rng.integers(0, B)] = ctx_max // size * size       # a full last block
    new[-1] = new_max
    width = int(max(-(-(c + n) // size) for c, n in zip(ctx, new))) + 2
    made = int(sum(-(-(c + n) // size) - -(-c // size) for c, n in zip(ctx, new)))
    pool = rng.permutation(made + 7 + B * width).astype(np.int32)
    head = 3
    free, table = pool[: made + head + 1], pool[made + 7:].reshape(B, width)     # held entries: any other ids
    t_max = int(new.sum()) + spare
    ws = workspace(512)
    st, got, _ = run_tables(ctx, new, size, free, head, table, t_max, ws)
    want = ref.build_tables(ctx, new, size, free, head, table, t_max)
    assert st == 0
    for key, w in zip(("table", "kv", "qo", "slots", "pos", "head"), want):
        np.testing.assert_array_equal(got[key], np.asarray(w).reshape(got[key].shape), err_msg=key)
    # the inputs are as they were: the same call again
    st, again, _ = run_tables(ctx, new, size, free, head, got["table"], t_max, ws)
    assert st == 0 and all(np.array_equal(again[k], got[k]) for k in got)


def test_tables_of_no_requests_and_no_tokens():
    ws = workspace(512)
    st, got, _ = run_tables([], [], 64, np.arange(4), 2, np.zeros((0, 4), np.int32), 5, ws)
    assert st == 0 and got["qo"].tolist() == [0] and got["head"].tolist() == [2] and (got["slots"] == -1).all()
    st, got, _ = run_tables([7, 0], [0, 0], 64, np.arange(4), 2, np.zeros((2, 4), np.int32), 0, ws)
    assert st == 0 and got["kv"].tolist() == [7, 0] and got["head"].tolist() == [2]


@pytest.mark.parametrize("what", ["negative length", "negative new", "too long", "too many tokens", "pool empty", "negative head"])
def test_tables_device_errors_write_nothing(what):
    ctx, new, free, head, t_max = [10, 70, 3], [1, 60, 1], np.arange(8), 0, 62
    if what == "negative length":
        ctx[1] = -1
    if what == "negative new":
        new[2] = -1
    if what == "too long":
        ctx[0] = 3 * 64
    if what == "too many tokens":
        t_max = 61
    if what == "pool empty":
        head = 8
    if what == "negative head":
        head = -1
    ws = workspace(512)
    st, _, same = run_tables(ctx, new, 64, free, head, np.full((3, 3), 5, np.int32), t_max, ws)
    assert st == moe.MOE_ERR_DEVICE_ASSERT and same
    assert status(ws) == 0                                 # reported once


# ------------------------------------------------------------------ append

def new_cache(blocks, heads, dim, size, rng):
    """A cache full of arbitrary bytes, with its guard bands and its mirror in 64 bits."""
    shapes = [(blocks, heads, size // 16, dim // 16, 16, 16), (blocks, heads, size // 16, dim, 16), (blocks, heads), (blocks, heads)]
    g = [Guarded(s, torch.uint8) for s in shapes]
    for x in g[:2]:
        x.t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(x.t.shape), dtype=np.uint8)))
    for x in g[2:]:
        x.t.copy_(torch.from_numpy(rng.integers(1, 247, tuple(x.t.shape), dtype=np.uint8)))
    return attn.KVCache(*[x.t for x in g]), g, ref.Cache.from_layout(*[x.t.cpu().numpy() for x in g])


def check_cache(g, mirror, label=""):
    for x, want, name in zip(g, mirror.layout(), ("k", "v", "k_scale", "v_scale")):
        x.check()
        np.testing.assert_array_equal(x.t.cpu().numpy(), want, err_msg=f"{label} {name}")


@pytest.mark.parametrize("heads,dim,size,lens", [
    (1, 64, 16, [1]), (8, 128, 64, [1, 1, 1]), (2, 128, 128, [300, 1, 128]), (3, 64, 32, [17, 2, 31, 64]), (2, 128, 16, [50, 16, 3]),
    (1, 128, 64, [700, 40])])
def test_append_matches_the_definition(heads, dim, size, lens):
    """Several steps into the same blocks, magnitudes that grow and shrink (so that held codes are
    re-rounded), from strided views; every byte of the cache is compared."""
    rng = np.random.default_rng(heads * dim + size)
    blocks = sum(-(-3 * n // size) + 1 for n in lens) + 2
    cache, g, mirror = new_cache(blocks, heads, dim, size, rng)
    order = rng.permutation(blocks)
    width, at, rows = max(-(-3 * n // size) for n in lens) + 1, 0, []
    for n in lens:
        rows.append(order[at: at + -(-3 * n // size)])
        at += len(rows[-1])
    ws = workspace(512)
    done = [0] * len(lens)
    for step in range(3):
        new = [n if step < 2 else max(1, n // 2) for n in lens]
        slots = np.concatenate([[int(rows[b][p // size]) * size + p % size for p in range(done[b], done[b] + n)] for b, n in enumerate(new)])
        T = len(slots)
        qkv = rng.standard_normal((T, 2 * heads + 1, dim)) * np.exp2(rng.integers(-12, 13, (T, 1, 1)) * (step + 1) / 2.0)
        if step == 0:
            qkv[:, :heads, :] *= 1e-3
        x = bf16(qkv)
        k, v = x[:, :heads], x[:, heads + 1:]
        attn.moe_kv_append(k, v, torch.from_numpy(slots).cuda(), cache, ws)
        assert status(ws) == 0
        mirror.append(f64(k), f64(v), slots)
        check_cache(g, mirror, f"step {step}")
        done = [d + n for d, n in zip(done, new)]


def test_append_special_values_and_skipped_tokens():
    rng = np.random.default_rng(5)
    cache, g, mirror = new_cache(4, 2, 64, 16, rng)
    x = rng.standard_normal((6, 4, 64)).astype(np.float32)
    x[0, 0, 3], x[0, 0, 4], x[0, 1, 5] = np.nan, np.inf, -np.inf
    x[0, 2] = 0.0                                           # a group of zeros only
    x[1, 2] = np.nan                                        # of nothing finite
    x[2] = 1e-39                                            # subnormal in bf16
    x[3] = 3.3e38                                           # near bf16's largest
    x[5, 0, 0] = -0.0
    slots = np.array([16, 17, -1, 32, 33, 48])
    ws = workspace(512)
    t = bf16(x)
    attn.moe_kv_append(t[:, :2], t[:, 2:], torch.from_numpy(slots).cuda(), cache, ws)
    assert status(ws) == 0
    mirror.append(f64(t[:, :2]), f64(t[:, 2:]), slots)
    check_cache(g, mirror)
    # zeros, then something larger: the zeros' exponent is the least one and grows
    attn.moe_kv_append(t[4:5, :2], t[4:5, 2:], torch.tensor([18]).cuda(), cache, ws)
    mirror.append(f64(t[4:5, :2]), f64(t[4:5, 2:]), np.array([18]))
    check_cache(g, mirror, "second")


def test_append_slot_outside_the_cache_is_skipped_and_reported():
    rng = np.random.default_rng(6)
    cache, g, mirror = new_cache(3, 1, 64, 32, rng)
    x = bf16(rng.standard_normal((3, 2, 64)))
    slots = np.array([32, 3 * 32, 64])
    ws = workspace(512)
    attn.moe_kv_append(x[:, :1], x[:, 1:], torch.from_numpy(slots).cuda(), cache, ws)
    assert status(ws) == moe.MOE_ERR_DEVICE_ASSERT
    mirror.append(f64(x[:, :1]), f64(x[:, 1:]), np.array([32, -1, 64]))
    check_cache(g, mirror)


def test_append_many_tokens_takes_the_windowed_launch():
    """More than 512 tokens: a CTA looks at 16 tokens; runs begin anywhere in a window."""
    rng = np.random.default_rng(7)
    cache, g, mirror = new_cache(200, 1, 64, 16, rng)
    lens = rng.integers(1, 30, 40)
    lens[3] = 250
    rows, at = [], 0
    order = rng.permutation(200)
    for n in lens:
        rows.append(order[at: at + -(-(n + 5) // 16)])
        at += len(rows[-1])
    assert at <= 200
    starts = rng.integers(0, 6, 40)
    slots = np.concatenate([[int(r[p // 16]) * 16 + p % 16 for p in range(s, s + n)] for r, s, n in zip(rows, starts, lens)])
    assert len(slots) > 512
    x = bf16(rng.standard_normal((len(slots), 2, 64)))
    ws = workspace(512)
    attn.moe_kv_append(x[:, :1], x[:, 1:], torch.from_numpy(slots).cuda(), cache, ws)
    assert status(ws) == 0
    mirror.append(f64(x[:, :1]), f64(x[:, 1:]), slots)
    check_cache(g, mirror)


# --------------------------------------------------------------- attention

class Problem:
    """Requests with (new, kv) tokens over a cache of random codes; slots past a
    request's length, and whole unused blocks, hold arbitrary bytes (NaN codes among them)."""

    def __init__(self, lens, kv_heads, group, dim, size, seed=0, exps=(-9, -5), q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.group, self.dim = rng, lens, group, dim
        self.n = [n for n, _ in lens]
        self.kv = [kv for _, kv in lens]
        need = [-(-kv // size) for kv in self.kv]
        blocks = sum(need) + 3
        width = max(need + [1]) + 1
        order = rng.permutation(blocks)
        table = np.full((len(lens), width), -7, np.int32)              # unused entries: not a block
        c = ref.Cache(blocks, kv_heads, dim, size)
        c.k[:], c.v[:] = rng.integers(0, 256, c.k.shape), rng.integers(0, 256, c.v.shape)
        c.ke[:], c.ve[:] = rng.integers(*exps, c.ke.shape, endpoint=True), rng.integers(*exps, c.ve.shape, endpoint=True)
        at = 0
        for b, kv in enumerate(self.kv):
            ids = order[at: at + need[b]]
            at += need[b]
            table[b, : len(ids)] = ids
            for i, p in enumerate(ids):                                # what is in use is finite
                live = min(size, kv - i * size)
                c.k[p, :, :live] = ref.e4m3_codes(np.clip(rng.standard_normal((kv_heads, live, dim)) * 90, -448, 448))
                c.v[p, :, :live] = ref.e4m3_codes(np.clip(rng.standard_normal((kv_heads, live, dim)) * 90, -448, 448))
        self.cache, self.table, self.size = c, table, size
        self.T = sum(self.n)
        self.offsets = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int64)
        heads = kv_heads * group
        self.qkv = bf16(rng.standard_normal((self.T, heads + 2, dim)) * q_scale)
        self.q = self.qkv[:, :heads]                                   # rows further apart than their heads
        self.scale = dim ** -0.5

    def run(self, causal=True, window=0, ws=None, table=None, offsets=None, kv=None, with_lse=True):
        dev = attn.KVCache(*[torch.from_numpy(a).cuda() for a in self.cache.layout()])
        heads = self.q.shape[1]
        out, lse = Guarded((self.T, heads, self.dim), torch.bfloat16), Guarded((self.T, heads), torch.float32)
        ws = workspace(attn.moe_kv_attention_workspace_size(max(self.T, 1), len(self.kv), heads, dev.kv_heads, self.dim)) if ws is None else ws
        attn.moe_kv_attention(self.q, dev, i32(self.table if table is None else table), i32(self.offsets if offsets is None else offsets),
                              i32(self.kv if kv is None else kv), self.scale, out.t, lse.t if with_lse else None, ws, causal=causal,
                              window=window)
        self.status = status(ws)
        out.check()
        lse.check()
        return out.t, lse.t

    def check(self, causal=True, window=0, **kw):
        out, lse = self.run(causal, window, **kw)
        assert self.status == 0
        want, want_lse, bound = ref.attention(f64(self.q), self.cache, self.table, self.offsets, self.kv, self.scale, causal, window)
        got, got_lse = f64(out), f64(lse)
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty) and not got[empty].any()
        err = np.abs(got - want)
        assert (err <= bound + 1e-30).all(), (float((err / (bound + 1e-30)).max()), np.argwhere(err > bound + 1e-30)[:4].tolist())
        d = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, want_lse))
        # scores of up to |x| in fp32: see the reference's bound; 2^-15 covers it for these inputs
        assert (d <= 2.0 ** -15 + 2.0 ** -20 * np.abs(np.where(empty, 0, want_lse))).all(), float(d.max())
        return out, lse


@pytest.mark.parametrize("size", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,kv_heads", [(1, 2), (5, 2), (8, 1), (16, 1), (20, 2)])
def test_attention_ragged_decode_and_verify(size, dim, group, kv_heads):
    lens = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 127), (1, 128), (1, 129), (2, 300), (4, 4), (3, 1000), (0, 50), (0, 0), (1, 257)]
    Problem(lens, kv_heads, group, dim, size, seed=size + group).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 16, 100, 5000])
def test_attention_masks(causal, window):
    p = Problem([(1, 400), (9, 40), (40, 300), (17, 17), (5, 3), (3, 0), (70, 333)], 2, 3, 64, 32, seed=window)
    p.check(causal, window)                                # (5, 3) and (3, 0): rows that see nothing


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_long_rows_and_many_tiles(dim):
    """Units of several row tiles, and one long request that all CTAs share."""
    Problem([(200, 900), (1, 40), (130, 130)], 2, 4, dim, 64, seed=3).check()
    Problem([(1, 9001)], 1, 8, dim, 16, seed=4).check()
    Problem([(3, 6000), (1, 2), (1, 5000)], 2, 12, dim, 128, seed=5).check()
    Problem([(2, 5000)], 1, 2, dim, 64, seed=6).check(window=4097)


def test_attention_peaked_scores():
    """Large scores: one key takes nearly all the weight."""
    Problem([(2, 700), (1, 64)], 2, 4, 128, 64, seed=8, q_scale=12.0).check()


def test_attention_block_exponents_far_apart():
    """Keys and values whose blocks differ by many binades, empty (all-zero) blocks among them."""
    p = Problem([(1, 500), (2, 260)], 2, 4, 64, 16, seed=9)
    rng = np.random.default_rng(10)
    p.cache.ve[:] = rng.integers(-60, 30, p.cache.ve.shape)
    p.cache.v[::3] = 0
    p.cache.ve[::3] = -126
    p.check()
    p.cache.ke[::4] = -126
    p.check()


def test_attention_q_range():
    """Rows of q of very different size, zeros among them."""
    p = Problem([(6, 200)], 1, 2, 64, 32, seed=11)
    f = torch.tensor([1e-20, 1.0, 0.0, 30.0, 1e-5, 2.0], device="cuda").view(6, 1, 1)
    p.qkv.copy_((p.qkv.float() * f).to(torch.bfloat16))
    p.check()


def test_attention_nan_reaches_only_rows_that_see_it():
    """A NaN among the values or keys of position 70 of 100, 40 new tokens (positions 60..99)."""
    for which in ("v", "k"):
        for window in (0, 8):
            p = Problem([(40, 100), (1, 90)], 1, 2, 64, 32, seed=12)
            clean_out, clean_lse = p.run(window=window)
            page = p.table[0, 70 // 32]
            getattr(p.cache, which)[page, 0, 70 % 32, 5] = 0x7F
            out, lse = p.run(window=window)
            assert p.status == 0
            pos = np.arange(60, 100)
            sees = (pos >= 70) & ((window == 0) | (70 > pos - window))
            o, co = out.float().cpu().numpy(), clean_out.float().cpu().numpy()
            assert np.array_equal(o[:40][~sees], co[:40][~sees]) and np.array_equal(o[40:], co[40:])
            if which == "v":
                assert np.isnan(o[:40][sees][..., 5]).all()
                keep = np.arange(64) != 5
                assert np.array_equal(o[:40][sees][..., keep], co[:40][sees][..., keep])
                assert torch.equal(lse, clean_lse)
            else:
                assert np.isnan(o[:40][sees]).all()


def test_attention_offsets_past_32_bits():
    """Blocks more than 4 GB into the cache."""
    p = Problem([(1, 100), (2, 40)], 8, 2, 128, 64, seed=13)
    k, v, ks, vs = p.cache.layout()
    blocks = (1 << 32) // (8 * 64 * 128) + 70
    dev = attn.KVCache.empty(blocks, 8, 128, 64)
    shift = blocks - k.shape[0]
    for t, a in zip((dev.k, dev.v, dev.k_scale, dev.v_scale), (k, v, ks, vs)):
        t[shift:] = torch.from_numpy(a).cuda()
    out, lse = torch.empty_like(p.q), torch.empty(p.q.shape[:2], device="cuda")
    out = torch.empty(p.q.shape, dtype=torch.bfloat16, device="cuda")
    ws = workspace()
    attn.moe_kv_attention(p.q, dev, i32(np.where(p.table >= 0, p.table + shift, -1)), i32(p.offsets), i32(p.kv), p.scale, out, lse, ws)
    assert status(ws) == 0
    want, want_lse = p.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # and the append there
    x = bf16(p.rng.standard_normal((1, 16, 128)))
    slots = torch.tensor([(blocks - 1) * 64 + 0]).cuda()
    attn.moe_kv_append(x[:, :8], x[:, 8:], slots, dev, ws)
    mirror = ref.Cache(1, 8, 128, 64)
    mirror.append(f64(x[:, :8]), f64(x[:, 8:]), np.array([0]))
    assert status(ws) == 0
    assert np.array_equal(dev.k[-1, :, 0, :, 0].cpu().numpy().reshape(8, 128), mirror.k[0, :, 0])
    assert np.array_equal(dev.v[-1, :, 0, :, 0].cpu().numpy(), mirror.v[0, :, 0])


def test_attention_repeats_bit_for_bit_and_without_lse():
    p = Problem([(1, 3000), (4, 700), (1, 20)], 4, 8, 128, 64, seed=14)
    a, la = p.run()
    b, lb = p.run()
    c, _ = p.run(with_lse=False)
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, c)


def test_attention_device_errors():
    p = Problem([(2, 100), (1, 50)], 1, 2, 64, 64, seed=15)
    sentinel = int(torch.full((1,), 0xA5A5, dtype=torch.int32).item())
    for bad in (dict(offsets=[0, 3, 2]), dict(offsets=[0, 2, 4]), dict(offsets=[-1, 2, 3]), dict(kv=[100, -1]), dict(kv=[100, 64 * 3 + 1])):
        out, _ = p.run(**bad)
        assert p.status == moe.MOE_ERR_DEVICE_ASSERT, bad
        assert (out.view(torch.int16).cpu().numpy().view(np.uint16) == sentinel).all()      # untouched
    table = p.table.copy()
    table[0, 0] = 1 << 20
    p.run(table=table)
    assert p.status == moe.MOE_ERR_DEVICE_ASSERT
    p.check()                                               # and the next call is well again


# -------------------------------------------------------------- projection

def linear_case(T, N, K, seed=0, x=None, ws=None):
    rng = np.random.default_rng(seed)
    if x is None:
        x = rng.standard_normal((T, K)) * np.exp2(rng.integers(-6, 7, (T, K // 16)).repeat(16, 1))
    big = bf16(np.concatenate([x, rng.standard_normal((T, 24))], 1))          # rows further apart than K
    xt = big[:, :K]
    w = bf16(rng.standard_normal((N, K)) * np.exp2(rng.integers(-8, 3, (N, 1))))
    weight = attn.FP8Weight.from_dense(w)
    y = Guarded((T, N), torch.bfloat16)
    ws = workspace(attn.moe_linear_fp8_workspace_size(T, N, K)) if ws is None else ws
    attn.moe_linear_fp8(xt, weight, y.t, ws)
    assert status(ws) == 0
    y.check()
    return xt, w, weight, y.t


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (200, 144), (129, 1040), (300, 4096)])
def test_weight_quantisation_matches_the_definition(N, K):
    rng = np.random.default_rng(N)
    x = rng.standard_normal((N, K)) * np.exp2(rng.integers(-20, 20, (1, K)))
    x[0, 0] = np.nan
    w = bf16(x)
    got = attn.FP8Weight.from_dense(w)
    d = f64(w)
    for r in range(-(-N // 128)):
        for c in range(-(-K // 128)):
            part = d[128 * r:128 * (r + 1), 128 * c:128 * (c + 1)]
            e = ref.least_exponent(ref.finite_max(part))
            assert got.scale[r, c].item() == e + 127
            np.testing.assert_array_equal(got.codes[128 * r:128 * (r + 1), 128 * c:128 * (c + 1)].cpu().numpy() & 0xFF,
                                          np.where(np.isnan(part), got.codes[128 * r:128 * (r + 1), 128 * c:128 * (c + 1)].cpu().numpy(),
                                                   ref.e4m3_codes(part / 2.0 ** e)))
    assert got.codes[0, 0].item() & 0x7F == 0x7F


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 192, 193, 500])
def test_linear_token_counts(T):
    xt, _, weight, y = linear_case(T, 333, 1040, seed=T)
    want, bound = ref.linear(f64(xt), weight.codes.cpu().numpy(), weight.scale.cpu().numpy())
    err = np.abs(f64(y) - want)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("N,K", [(1, 16), (7, 48), (128, 128), (129, 2048), (1000, 16), (2, 8192), (3000, 512)])
@pytest.mark.parametrize("T", [1, 40, 200])
def test_linear_shapes(T, N, K):
    xt, _, weight, y = linear_case(T, N, K, seed=N + K)
    want, bound = ref.linear(f64(xt), weight.codes.cpu().numpy(), weight.scale.cpu().numpy())
    err = np.abs(f64(y) - want)
    assert (err <= bound).all(), float((err / bound).max())


def test_linear_special_rows_stay_apart():
    """A token of zeros gives zeros, one that is not finite gives NaN, and neither touches the others."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 256))
    clean = linear_case(20, 300, 256, seed=4, x=x)[3]
    x2 = x.copy()
    x2[3], x2[7, 10], x2[11, 200] = 0.0, np.inf, np.nan
    y = linear_case(20, 300, 256, seed=4, x=x2)[3]
    keep = [i for i in range(20) if i not in (3, 7, 11)]
    assert torch.equal(y[keep], clean[keep])
    assert not y[3].any() and torch.isnan(y[[7, 11]].float()).all()


@pytest.mark.parametrize("T", [1, 150, 600])
def test_linear_repeats_bit_for_bit(T):
    ws = workspace(attn.moe_linear_fp8_workspace_size(T, 1111, 2064))
    a = linear_case(T, 1111, 2064, seed=1, ws=ws)[3].clone()
    b = linear_case(T, 1111, 2064, seed=1, ws=ws)[3]
    assert torch.equal(a, b)


# ------------------------------------------------------------ a whole step

def step(state, ws, stream=None):
    s = state
    attn.moe_kv_build_tables(s["ctx"], s["new"], 32, s["free"], s["head"], s["table"], s["kv"], s["qo"], s["slots"], s["pos"], s["head_out"],
                             ws, stream)
    attn.moe_linear_fp8(s["x"], s["w"], s["qkv"].view(s["T"], -1), ws, stream)
    attn.moe_kv_append(s["qkv"][:, 8:10], s["qkv"][:, 10:], s["slots"], s["cache"], ws, stream)
    attn.moe_kv_attention(s["qkv"][:, :8], s["cache"], s["table"], s["qo"], s["kv"], 0.125, s["out"], s["lse"], ws, stream=stream)


def new_state(seed=0):
    rng = np.random.default_rng(seed)
    ctx, new = [40, 0, 100, 31], [1, 9, 2, 1]
    T = sum(new)
    pool = rng.permutation(40)
    table = np.full((4, 6), -1)
    at = 0
    for b, c in enumerate(ctx):
        n = -(-c // 32)
        table[b, :n] = pool[at: at + n]
        at += n
    cache = attn.KVCache.empty(40, 2, 64, 32)
    for t in (cache.k, cache.v):
        t.copy_(torch.from_numpy(ref.e4m3_codes(np.clip(rng.standard_normal(tuple(t.shape)) * 90, -448, 448))))
    cache.k_scale.fill_(120)
    cache.v_scale.fill_(120)
    dev = dict(device="cuda")
    return dict(T=T, ctx=i32(ctx), new=i32(new), free=i32(pool[at:]), head=i32([0]), head_out=i32([0]), table=i32(table),
                kv=torch.zeros(4, dtype=torch.int32, **dev), qo=torch.zeros(5, dtype=torch.int32, **dev),
                slots=torch.zeros(T, dtype=torch.int64, **dev), pos=torch.zeros(T, dtype=torch.int32, **dev),
                x=bf16(rng.standard_normal((T, 256))), w=attn.FP8Weight.from_dense(bf16(rng.standard_normal((12 * 64, 256)) / 16)),
                qkv=torch.zeros(T, 12, 64, dtype=torch.bfloat16, **dev), cache=cache,
                out=torch.zeros(T, 8, 64, dtype=torch.bfloat16, **dev), lse=torch.zeros(T, 8, **dev))


def results(s):
    return [s[k].clone() for k in ("table", "kv", "qo", "slots", "pos", "head_out", "qkv", "out", "lse")] + [s["cache"].k.clone(),
                                                                                                          s["cache"].v.clone()]


def test_step_against_the_reference():
    s, ws = new_state(), workspace()
    mirror = ref.Cache.from_layout(*[t.cpu().numpy() for t in (s["cache"].k, s["cache"].v, s["cache"].k_scale, s["cache"].v_scale)])
    step(s, ws)
    assert status(ws) == 0
    qkv = f64(s["qkv"])
    mirror.append(qkv[:, 8:10], qkv[:, 10:], s["slots"].cpu().numpy())
    want, want_lse, bound = ref.attention(qkv[:, :8], mirror, s["table"].cpu().numpy(), s["qo"].tolist(), s["kv"].tolist(), 0.125)
    assert (np.abs(f64(s["out"]) - want) <= bound).all()
    assert np.abs(f64(s["lse"]) - want_lse).max() < 2.0 ** -13


def test_step_on_a_side_stream_and_in_a_graph():
    s, ws = new_state(), workspace()
    step(s, ws)
    want = results(s)
    side = torch.cuda.Stream()
    t = new_state()
    side.wait_stream(torch.cuda.current_stream())
    step(t, ws, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results(t)))
    u = new_state()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(u, ws)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results(u)))
    g.replay()                                              # the step repeats: same tables, same codes
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results(u)))
    assert status(ws) == 0


def test_workspace_is_shared_with_the_moe_layer():
    """The attention's regions and the MoE layer's take turns in one workspace."""
    from block_scaled_fp4_moe_gb300 import inputs
    from gpu_support import Problem as MoEProblem
    p = MoEProblem.from_config(inputs.CONFIGS["tiny"])
    want = p.forward()
    ws = workspace()
    s = new_state()
    step(s, ws)
    first = results(s)
    got = p.forward(ws)
    assert np.array_equal(got["y"], want["y"]) and np.array_equal(got["ids"], want["ids"])
    step(s, ws)
    assert status(ws) == 0 and all(torch.equal(a, b) for a, b in zip(first, results(s)))


def test_binding_refusals():
    p = Problem([(1, 20)], 2, 2, 64, 16)
    dev = attn.KVCache(*[torch.from_numpy(a).cuda() for a in p.cache.layout()])
    out, ws = torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda"), workspace()
    args = dict(q=p.q, cache=dev, block_table=i32(p.table), q_offsets=i32([0, 1]), kv_lens=i32([20]), softmax_scale=0.1, out=out, lse=None,
                ws=ws)
    attn.moe_kv_attention(**args)
    for bad in (dict(q=p.q.float()), dict(q=p.q.cpu()), dict(out=out[:, :2]), dict(q_offsets=i32([0])), dict(block_table=i32(p.table).long()),
                dict(kv_lens=i32([20, 1]))):
        with pytest.raises(ValueError):
            attn.moe_kv_attention(**{**args, **bad})
    with pytest.raises(moe.MoEError):
        attn.moe_kv_attention(**{**args, "ws": torch.zeros(1024, dtype=torch.uint8, device="cuda")})
    with pytest.raises(ValueError):
        attn.KVCache(dev.k, dev.k, dev.k_scale, dev.v_scale)
    w = attn.FP8Weight.from_dense(bf16(np.ones((16, 32))))
    with pytest.raises(ValueError):
        attn.moe_linear_fp8(bf16(np.ones((2, 16))), w, torch.empty(2, 16, dtype=torch.bfloat16, device="cuda"), ws)
    with pytest.raises(ValueError):
        attn.FP8Weight(w.codes, w.scale[:0])


# ------------------------------------- units of many rows (tensor-memory form)

@pytest.mark.parametrize("dim,size", [(64, 32), (128, 16), (128, 128), (64, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 130), (False, 33)])
def test_attention_many_rows(dim, size, causal, window):
    """More than 24 rows a request and 64 units: row tiles of 1 .. 256 rows, one half or two, requests that see nothing, a cut
    last tile, a request without new tokens."""
    lens = [(30, 300), (1, 129), (64, 64), (17, 515), (0, 40), (9, 3), (100, 260), (33, 640), (5, 128)]
    Problem(lens, 8, 8, dim, size, seed=dim + size).check(causal, window)


def test_attention_many_rows_cut_into_pieces():
    """Fewer units than CTAs: every unit lies in several, with one or both halves in each."""
    Problem([(30, 6000)], 8, 8, 64, 64, seed=31).check()
    Problem([(8, 5000)] * 8, 8, 4, 128, 16, seed=32).check()
    Problem([(8, 300 + 17 * i) for i in range(9)], 8, 6, 64, 128, seed=33).check(window=200)


def test_attention_many_rows_ranges():
    """Block exponents far apart, rows of q of very different size, scores that grow along the cache."""
    p = Problem([(12, 400), (12, 300)] * 5, 8, 4, 64, 16, seed=34)
    rng = np.random.default_rng(35)
    p.cache.ve[:] = rng.integers(-60, 30, p.cache.ve.shape)
    p.cache.v[::3] = 0
    p.cache.ve[::3] = -126
    p.check()
    p = Problem([(12, 700)] * 10, 8, 4, 128, 64, seed=36, q_scale=6.0)
    p.cache.ke[:] = np.sort(rng.integers(-12, -4, p.cache.ke.shape), axis=0)
    p.check()


def test_attention_many_rows_nan_reaches_only_rows_that_see_it():
    for which in ("v", "k"):
        for window in (0, 8):
            p = Problem([(40, 200), (33, 90), (20, 130)] * 4, 8, 4, 64, 32, seed=37)
            clean_out, clean_lse = p.run(window=window)
            page = p.table[0, 170 // 32]
            getattr(p.cache, which)[page, 1, 170 % 32, 5] = 0x7F
            out, lse = p.run(window=window)
            assert p.status == 0
            pos = np.arange(160, 200)
            sees = (pos >= 170) & ((window == 0) | (170 > pos - window))
            o, co = out.float().cpu().numpy(), clean_out.float().cpu().numpy()
            hit = slice(4, 8)                              # the query heads of key/value head 1
            assert np.array_equal(o[40:], co[40:]) and np.array_equal(o[:40, :4], co[:40, :4]) and np.array_equal(o[:40, 8:], co[:40, 8:])
            assert np.array_equal(o[:40, hit][~sees], co[:40, hit][~sees])
            if which == "v":
                keep = np.arange(64) != 5
                assert np.isnan(o[:40, hit][sees][..., 5]).all()
                assert np.array_equal(o[:40, hit][sees][..., keep], co[:40, hit][sees][..., keep]) and torch.equal(lse, clean_lse)
            else:
                assert np.isnan(o[:40, hit][sees]).all()


def test_attention_many_rows_repeats_bit_for_bit():
    p = Problem([(30, 2000), (64, 900), (40, 40)], 8, 8, 128, 64, seed=38)
    a, la = p.run()
    b, lb = p.run()
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dim,size,seed", [(64, 32, 39), (128, 16, 40), (128, 64, 41)])
def test_attention_many_rows_whole_units_beside_cut_ones(dim, size, seed):
    """A CTA's range holds whole units of two and more tiles (both halves work on the same rows) between parts of others."""
    p = Problem([(8, 9000)] + [(8, 150 + 70 * i) for i in range(9)], 8, 4, dim, size, seed=seed)
    a, la = p.check()
    b, lb = p.run()
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("kv_heads,group,dim,lens", [
    (2, 1, 128, [(1, 2516), (1, 1623)]), (2, 3, 128, [(1, 18298)]), (2, 4, 64, [(1, 3609)]), (1, 1, 64, [(1, 9000)]), (1, 1, 128, [(1, 1)]),
    (8, 5, 128, [(1, 1000)]), (4, 4, 64, [(14, 5000)]), (8, 1, 64, [(1, 900 * i + 1) for i in range(6)]), (2, 16, 128, [(3, 7000)]),
    (8, 4, 128, [(8, 5000)] * 8), (8, 1, 64, [(26, 800 * i + 30) for i in range(9)])])
def test_attention_few_rows_cut_into_many_parts(kv_heads, group, dim, lens):
    """Fewer rows than a unit's: their parts lie close together in a workspace of just the size asked for, and none past its end."""
    p = Problem(lens, kv_heads, group, dim, 32, seed=42)
    n = attn.moe_kv_attention_workspace_size(p.T, len(lens), kv_heads * group, kv_heads, dim)
    guarded = torch.full((n + (1 << 24),), 0xA5, dtype=torch.uint8, device="cuda")
    guarded[:n] = 0
    p.check(ws=guarded[:n])
    p.check(causal=False, window=700, ws=guarded[:n])
    assert bool((guarded[n:] == 0xA5).all())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("step,q_scale", [(1, 1.0), (3, 4.0), (-2, 4.0)])
def test_attention_many_rows_references_move_inside_a_tile(dim, step, q_scale):
    """Key exponents that climb (or fall) from block to block of 16 tokens, eight to a tile, and values' exponents against them."""
    p = Problem([(9, 700), (9, 130)] * 5, 8, 4, dim, 16, seed=43, q_scale=q_scale)
    for row, kv in zip(p.table, p.kv):
        for i in range(-(-kv // 16)):
            p.cache.ke[row[i]] = -14 + step * (i % 11)
            p.cache.ve[row[i]] = -3 * step * (i % 7)
    p.check()


@pytest.mark.parametrize("T", [1, 8, 40])
def test_linear_directly_after_its_weights(T):
    """Weights written by the kernel just before, the library's own or another, are the ones that the product reads."""
    N, K = 4096, 7168
    rng = np.random.default_rng(44)
    x = bf16(rng.standard_normal((T, K)))
    dense = [torch.randn(N, K, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    w = [attn.FP8Weight.from_dense(d) for d in dense]
    ws = workspace(attn.moe_linear_fp8_workspace_size(T, N, K))
    want = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for i in range(2):
        attn.moe_linear_fp8(x, w[i], want[i], ws)
    torch.cuda.synchronize()
    one = attn.FP8Weight(w[0].codes.clone(), w[0].scale.clone())
    got = [torch.empty_like(want[0]) for _ in range(40)]
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        if i % 4 < 2:
            attn.moe_quantize_fp8_weight(dense[i % 2], one)
        else:
            one.codes.copy_(w[i % 2].codes)
            one.scale.copy_(w[i % 2].scale)
        attn.moe_linear_fp8(x, one, y, ws)
    torch.cuda.synchronize()
    assert [i for i, y in enumerate(got) if not torch.equal(y, want[i % 2])] == []


@pytest.mark.parametrize("causal", [True, False])
def test_attention_widest_window(causal):
    """The largest window a call can name, with requests that bring more tokens than the cache holds of them."""
    Problem([(9, 3), (4, 200), (1, 1)], 2, 4, 64, 16, seed=45).check(causal, 2 ** 31 - 1)
    Problem([(40, 30), (30, 200), (30, 3)] * 2, 8, 8, 128, 16, seed=46).check(causal, 2 ** 31 - 1)


def test_single_token_strides_do_not_matter():
    """A lone token's, or head's, stride is not used: whatever a view gives is taken."""
    p = Problem([(1, 77)], 1, 1, 64, 16, seed=47)
    want, want_lse = p.check()
    p.q = p.q.contiguous().as_strided((1, 1, 64), (3, 5, 1))
    got, lse = p.check()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    x, w = bf16(np.random.default_rng(48).standard_normal((1, 64))), attn.FP8Weight.from_dense(bf16(np.eye(64)))
    ws = workspace()
    y = [torch.empty(1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    attn.moe_linear_fp8(x, w, y[0], ws)
    attn.moe_linear_fp8(x.as_strided((1, 64), (7, 1)), w, y[1], ws)
    assert torch.equal(*y)


@pytest.mark.parametrize("dim,new,group", [(64, 60, 4), (64, 9, 4), (128, 40, 8), (128, 7, 4), (64, 120, 2), (128, 60, 4), (128, 30, 4)])
def test_attention_many_rows_many_nan_values(dim, new, group):
    """Every value of 45 consecutive tokens among the newest is NaN: all rows that see one of them are, and no other."""
    kv, first = 400, 400 - new // 2 - 1                   # some new tokens come before them, and see none
    p = Problem([(new, kv)] * 5, 8, group, dim, 32, seed=49)
    clean_out, clean_lse = p.run()
    for b in range(5):
        for j in range(first, min(first + 45, kv)):
            p.cache.v[p.table[b, j // 32], :, j % 32] = 0x7F
    out, lse = p.run()
    assert p.status == 0 and torch.equal(lse, clean_lse)
    sees = torch.tensor([kv - new + i >= first for i in range(new)] * 5, device="cuda")
    assert sees.any() and not sees.all()
    assert torch.equal(out[~sees], clean_out[~sees]) and bool(torch.isnan(out[sees].float()).all())


@pytest.mark.parametrize("T,N,K", [(1, 40000, 144), (9, 40001, 128), (100, 40000, 16), (128, 21000, 272), (130, 16500, 128), (300, 7000, 256), (400, 7000, 256),
                                   (650, 7000, 128)])
def test_linear_forms_by_size(T, N, K):
    """More tiles than SMs, with one token tile and with several; tiles that share an SM; a grid that walks."""
    xt, _, weight, y = linear_case(T, N, K, seed=50)
    want, bound = ref.linear(f64(xt), weight.codes.cpu().numpy(), weight.scale.cpu().numpy())
    assert (np.abs(f64(y) - want) <= bound).all()


@pytest.mark.parametrize("dim,new,group,kv,nans", [(128, 20, 4, 100, 15), (128, 20, 4, 230, 15), (64, 20, 4, 120, 15), (64, 30, 2, 250, 24),
                                                   (128, 8, 8, 60, 6), (128, 100, 4, 128, 40)])
def test_attention_many_rows_nan_values_of_unit_after_unit(dim, new, group, kv, nans):
    """More units than CTAs, of one or two tiles each and of one request or another: the NaN values of every head and request are found
    by their own rows alone, also where the next unit's are met meanwhile and where there are more than a CTA's list holds."""
    B, first = 60, kv - new // 2 - 1                      # some new tokens come before the NaN ones, and see none
    p = Problem([(new, kv - b % 3) for b in range(B)], 8, group, dim, 32, seed=51)
    clean_out, clean_lse = p.run()
    sees = []
    for b in range(B):
        end = min(first + nans, p.kv[b])
        has = b % 4 != 3                                   # some requests have none
        for j in range(first, end if has else first):
            p.cache.v[p.table[b, j // 32], :, j % 32] = 0x7F
        sees += [has and p.kv[b] - new + i >= first for i in range(new)]
    out, lse = p.run()
    sees = torch.tensor(sees, device="cuda")
    assert p.status == 0 and torch.equal(lse, clean_lse) and sees.any() and not sees.all()
    assert torch.equal(out[~sees], clean_out[~sees]) and bool(torch.isnan(out[sees].float()).all())
    again, _ = p.run()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("size", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,kv_heads,group,lens", [
    (64, 2, 4, [(1, 700), (2, 300), (1, 90), (3, 129)]), (128, 1, 8, [(1, 700), (2, 300), (1, 90), (4, 257)]), (128, 2, 8, [(8, 500), (7, 200)]),
    (64, 8, 4, [(9, 700), (20, 300), (40, 200), (8, 90)]), (128, 8, 8, [(40, 700), (9, 300), (30, 260), (12, 130)])])
def test_attention_blocks_before_the_window_are_not_looked_at(size, dim, kv_heads, group, lens):
    """Entries of blocks that no row sees any more may be anything, and so may what lies before the window in a block that is seen."""
    for window in (1, 20, 100, 150):
        p = Problem(lens, kv_heads, group, dim, size, seed=52)
        want, want_lse = p.check(window=window)
        table = p.table.copy()
        for b, (n, kv) in enumerate(lens):
            first = max(0, kv - n - window + 1)            # the first new token's first position
            table[b, : first // size] = -1
            if first % size:
                block = p.table[b, first // size]
                p.cache.k[block, :, : first % size] = 0x7F
                p.cache.v[block, :, : first % size] = 0xFF
        got, lse = p.run(window=window, table=table)
        assert p.status == 0
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("B", [4053, 4054, 4095, 4096])
def test_tables_of_the_batches_around_48_kb_of_shared_memory(B):
    """In a process of their own: a larger batch before them would have raised the kernel's limit for them."""
    code = f"import test_gpu_attn as t; t.test_tables_match_the_definition({B}, 16, 40, 2, 5)"
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", code], cwd=here, env={**os.environ, "PYTHONPATH": os.path.dirname(here)}, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


LONG_KERNEL = r"""
#include <cstdint>
// Lets the next kernel start at once, and runs for `ms` more on one SM.
__global__ void long_kernel(unsigned ms) {
    asm volatile("griddepcontrol.launch_dependents;");
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    for (unsigned i = 0; i < 1000u * ms; ++i) {            // at most 1 us each: ends by itself whatever the timer says
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t - t0 > ms * 1000000ull)
            break;
    }
}
extern "C" int run_long_kernel(unsigned ms, void *stream) {
    long_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(ms);
    return cudaGetLastError();
}
"""


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_linear_behind_a_kernel_that_runs_for_long(T, tmp_path):
    """The limits of a call's waits do not count what the kernel before it still has to do."""
    src, lib = tmp_path / "long.cu", tmp_path / "long.so"
    src.write_text(LONG_KERNEL)
    subprocess.run([_build.nvcc_path(), *_build.ARCH_FLAGS, "-shared", "-Xcompiler", "-fPIC", "-o", str(lib), str(src)], check=True)
    run = ctypes.CDLL(str(lib)).run_long_kernel
    run.argtypes = [ctypes.c_uint, ctypes.c_void_p]
    ws = workspace(attn.moe_linear_fp8_workspace_size(T, 333, 1040))
    xt, _, weight, want = linear_case(T, 333, 1040, seed=53, ws=ws)
    y = torch.zeros_like(want)
    assert run(400, torch.cuda.current_stream().cuda_stream) == 0
    attn.moe_linear_fp8(xt, weight, y, ws)
    torch.cuda.synchronize()
    assert status(ws) == 0 and torch.equal(y, want)


@pytest.mark.parametrize("dim,group,new", [(64, 4, 9), (128, 4, 9), (128, 20, 13), (64, 5, 1), (128, 8, 3)])
def test_attention_with_a_window_does_not_depend_on_other_requests(dim, group, new):
    """Every other request's keys are NaN, or not: where a tile begins with blocks that are not read, what the CTA read before lies there, and has no
    part in the bits.  (A window's first tile has larger keys and smaller values than the others: the references of rows with tokens stay, those of
    the unit's rows without, whose scores are zero, would not.)"""
    window, lens = 425, [(new, 600 + 37 * (i % 12)) for i in range(300)]
    p = Problem(lens, 1, group, dim, 16, seed=69, exps=(-7, -7))
    p.cache.ve[:] = 2
    for row, (n, kv) in zip(p.table, lens):
        first = row[: ((kv - n - window + 1) // 128 + 1) * 8]
        p.cache.ke[first], p.cache.ve[first] = -5, -8
    want, want_lse = p.run(window=window)
    assert p.status == 0
    p.cache.k[p.table[::2, : 600 // 16]] = 0x7F
    out, lse = p.run(window=window)
    assert p.status == 0
    t = torch.arange(p.T, device="cuda") // new % 2 == 1
    assert bool(torch.isnan(lse[~t]).all()) and torch.equal(out[t], want[t]) and torch.equal(lse[t], want_lse[t])
