"""Norm, rotary positions, latent append and latent attention on the GPU against their definitions in 64 bits, within bounds derived
from the kernels' arithmetic (layer_ops_reference)."""
import math

import numpy as np
import pytest
import torch

import layer_ops_reference as ref
from block_scaled_fp4_moe_gb300 import _build, attn, moe
from test_gpu_attn_forms import has, kernels

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


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


def within(got, want, bound, what=""):
    err = (got.double() - want).abs()
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound, at {np.unravel_index(int((err / bound).argmax()), err.shape)}"


# -------------------------------------------------------------------- norm

@pytest.mark.parametrize("T,H", [(1, 8), (3, 64), (5, 256), (9, 264), (61, 512), (7, 1024), (2, 1032), (33, 5120), (200, 7168), (3, 8192), (2, 8200),
                                 (2, 16384), (1, 32768), (500, 40)])
@pytest.mark.parametrize("form", ["norm", "residual", "wide", "gated", "rows", "post", "all"])
def test_norm_matches_the_definition(T, H, form):
    g = gen(T * 1000 + H)
    x = normal(g, T, H + 24)[:, :H] if form != "norm" else normal(g, T, H)       # rows further apart
    x[:, :: 61] *= 12
    wide = form in ("wide", "all")
    res = None if form == "norm" else normal(g, T, H, std=3.0, dtype=torch.float32 if wide else torch.bfloat16)
    post = 1 + normal(g, H, std=0.2) if form in ("post", "all") else None
    gate = normal(g, H) if form == "gated" else normal(g, T, H + 8)[:, :H] if form in ("rows", "all") else None
    weight, scale, eps = 1 + normal(g, H, std=0.2), 1.0 if form in ("norm", "residual") else -0.37, 1e-5
    y, out = Guarded((T, H), torch.bfloat16), Guarded((T, H), torch.float32 if wide else torch.bfloat16)
    attn.moe_rms_norm(x, weight, eps, y.t, residual=res, residual_out=out.t if res is not None else None, post_weight=post, gate=gate, scale=scale)
    y.check(), out.check()
    # the call rounds its scalars to fp32
    want, bound, h, h_bound = ref.rms_norm(x, float(np.float32(eps)), weight, res, post, gate, float(np.float32(scale)), wide)
    within(y.t, want, bound, "y")
    if res is not None:
        within(out.t, h, h_bound, "h")
        again = torch.empty_like(y.t)                      # in place, and h alone: the same bits
        kept, only, x2 = res.clone(), torch.empty_like(res), x.clone() if x.is_contiguous() else x
        attn.moe_rms_norm(x, weight, eps, again, residual=kept, residual_out=kept, post_weight=post, gate=gate, scale=scale)
        attn.moe_rms_norm(x, None, eps, None, residual=res, residual_out=only, post_weight=post, gate=gate, scale=scale)
        assert torch.equal(again, y.t) and torch.equal(kept, out.t) and torch.equal(only, out.t)
    else:
        x2 = x.clone()
        attn.moe_rms_norm(x2, weight, eps, x2)             # y over x
        assert torch.equal(x2, y.t)


def test_norm_of_rows_that_are_not_finite_leaves_the_others():
    g = gen(3)
    x, r, w = normal(g, 6, 2048), normal(g, 6, 2048), normal(g, 2048)
    clean, out = torch.empty_like(x), torch.empty_like(x)
    attn.moe_rms_norm(x, w, 1e-6, clean, residual=r)
    x[1, 5], x[3, 2000], r[4, 7] = math.nan, math.inf, -math.inf
    attn.moe_rms_norm(x, w, 1e-6, out, residual=r)
    keep = torch.tensor([0, 2, 5], device="cuda")
    assert torch.equal(out[keep], clean[keep])
    assert out[1].isnan().all() and out[3, 2000].isnan() and out[4, 7].isnan()
    assert (out[3, :2000] == 0).all() and (out[4, 8:] == 0).all()      # the rest over an infinite root
    zero = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(zero, 7.0)
    attn.moe_rms_norm(zero, w[:64], 1e-6, y)
    assert (y == 0).all()


def test_norm_of_no_tokens():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    attn.moe_rms_norm(e, torch.ones(64, dtype=torch.bfloat16, device="cuda"), 1e-6, e)


# ------------------------------------------------------------------ rotary

CASES = [  # D, pairs, offset, heads, kv_heads
    (16, 8, 0, 1, 0), (64, 32, 0, 4, 1), (128, 64, 0, 64, 8), (128, 32, 64, 40, 8), (128, 32, 0, 5, 3), (192, 32, 128, 16, 0), (256, 128, 0, 3, 2),
    (96, 24, 16, 7, 1), (200, 8, 184, 2, 2), (64, 8, 24, 128, 4)]


@pytest.mark.parametrize("D,pairs,offset,hq,hk", CASES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("T", [1, 9, 700])
def test_rotary_matches_the_definition(D, pairs, offset, hq, hk, inter, normed, T):
    if T == 700 and hq * D > 1024:
        T = 610                                            # a CTA for a token, whatever its heads
    g = gen(D + pairs + T)
    qkv = normal(g, T, hq + 2 * hk + 1, D)
    table = attn.RotaryTable.make(2 * pairs, scaling="parts" if normed else None, factor=4.0 if normed else 1.0, original_len=4096)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").to(torch.int32)
    if T > 1:
        pos[0], pos[1] = 0, 2 ** 31 - 1
        pos[-1] = -1                                       # behind the last token
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    qn, kn = (1 + normal(g, D, std=0.2), 1 + normal(g, D, std=0.2)) if normed else (None, None)
    amp = float(np.float32(table.amplitude))
    live = pos >= 0
    out = [Guarded((T, h, D), torch.bfloat16) for h in (hq, hk)]
    before = [o.t.clone() for o in out]
    extra = dict(k=k, k_out=out[1].t, k_norm=kn) if hk else {}
    attn.moe_rotary(q, pos, table, out[0].t, interleaved=inter, offset=offset, q_norm=qn, eps=1e-6, **extra)
    for x, w, o, b in ((q, qn, out[0], before[0]), (k, kn, out[1], before[1])):
        o.check()
        if x.shape[1]:
            want, bound = ref.rotary(x[live], pos[live], table.turns, amp, inter, offset, w, float(np.float32(1e-6)))
            within(o.t[live], want, bound)
            assert torch.equal(o.t[~live].view(torch.int16), b[~live].view(torch.int16))
            if w is None:                                  # dims that are not rotated are copied
                assert torch.equal(o.t[live][..., :offset], x[live][..., :offset])
                assert torch.equal(o.t[live][..., offset + 2 * pairs:], x[live][..., offset + 2 * pairs:])
    # in place, on views of the projection's output: the same bits, and nothing else is touched
    mine = qkv.clone()
    extra = dict(k=mine[:, hq:hq + hk], k_out=mine[:, hq:hq + hk], k_norm=kn) if hk else {}
    attn.moe_rotary(mine[:, :hq], pos, table, mine[:, :hq], interleaved=inter, offset=offset, q_norm=qn, eps=1e-6, **extra)
    assert torch.equal(mine[live][:, :hq], out[0].t[live]) and torch.equal(mine[live][:, hq:hq + hk], out[1].t[live])
    assert torch.equal(mine[:, hq + hk:], qkv[:, hq + hk:]) and torch.equal(mine[~live], qkv[~live])


def test_rotary_of_other_strides_and_of_no_tokens():
    g = gen(5)
    wide = normal(g, 6, 3, 2, 64)
    q, out = wide[:, :, 0], torch.zeros(3, 6, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)     # heads outermost
    table, pos = attn.RotaryTable.make(64), i32([5, 4, 3, 2, 1, 0])
    attn.moe_rotary(q, pos, table, out)
    want, bound = ref.rotary(q, pos, table.turns)
    within(out, want, bound)
    e = torch.empty(0, 3, 64, dtype=torch.bfloat16, device="cuda")
    attn.moe_rotary(e, i32([]), table, e)


def test_rotary_keeps_dot_products_of_equal_distances():
    """What it is for: q.k depends on the distance alone, here a million positions out."""
    g = gen(6)
    v = normal(g, 1, 2, 128).expand(2, 2, 128).contiguous()
    table = attn.RotaryTable.make(128)
    dots = []
    for base in (3, 1_000_003):
        out = torch.empty_like(v)
        attn.moe_rotary(v, i32([base, base + 17]), table, out)
        dots.append((out[0].double() * out[1].double()).sum(-1))
    # both sides round 128 products of values of bf16: 2 * 2^-8 of the sum of magnitudes
    assert ((dots[0] - dots[1]).abs() <= 4 * ref.U16 * (v[0].double() ** 2).sum(-1)).all()


# ----------------------------------------------------------- latent append

@pytest.mark.parametrize("T,latent,block", [(1, 512, 64), (3, 256, 16), (64, 512, 128), (333, 512, 32), (1201, 256, 64)])
@pytest.mark.parametrize("form", ["plain", "halves", "neighbours"])
def test_latent_append_matches_the_definition(T, latent, block, form):
    g = gen(T + latent)
    nb = -(-T // block) + 5
    both = normal(g, T, latent + 64 + 8, std=2.0)
    c, k = both[:, :latent], both[:, latent:latent + 64]
    slots = torch.randperm(nb * block, generator=g, device="cuda")[:T].clone()
    if T > 2:
        slots[T // 2] = -1
    data = Guarded((nb, block, latent + 64), torch.bfloat16)
    before = data.t.clone()
    cache, ws = attn.LatentCache(data.t), torch.zeros(512, dtype=torch.uint8, device="cuda")
    norm = 1 + normal(g, latent, std=0.2) if form != "plain" else None
    table, pos = attn.RotaryTable.make(64), torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").to(torch.int32)
    extra = {} if form == "plain" else dict(positions=pos, table=table, interleaved=form == "neighbours")
    attn.moe_latent_append(c, k, slots, cache, ws, norm=norm, eps=1e-6, **extra)
    assert moe.moe_check_device_status(ws) == 0
    data.check()
    live = slots >= 0
    rows, at = data.t.view(-1, latent + 64), slots[live]
    if form == "plain":
        assert torch.equal(rows[at], torch.cat((c, k), 1)[live])
    else:
        want, bound, _, _ = ref.rms_norm(c, float(np.float32(1e-6)), norm)
        within(rows[at][:, :latent], want[live], bound[live], "latent")
        want, bound = ref.rotary(k[live][:, None], pos[live], table.turns, 1.0, form == "neighbours")
        within(rows[at][:, latent:], want[:, 0], bound[:, 0], "key")
    rest = torch.ones(nb * block, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(rows[rest].view(torch.int16), before.view(-1, latent + 64)[rest].view(torch.int16))


def test_latent_append_past_the_cache_is_left_out_and_reported():
    g = gen(8)
    c, k = normal(g, 3, 256), normal(g, 3, 64)
    data = Guarded((2, 16, 320), torch.bfloat16)
    before, ws = data.t.clone(), torch.zeros(512, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([31, 32, 1 << 40], device="cuda")
    attn.moe_latent_append(c, k, slots, attn.LatentCache(data.t), ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_ASSERT
    data.check()
    assert torch.equal(data.t[1, 15], torch.cat((c, k), 1)[0])
    assert torch.equal(data.t.view(32, 320)[:31].view(torch.int16), before.view(32, 320)[:31].view(torch.int16))


# -------------------------------------------------------- latent attention

class Step:
    """Requests with kv tokens, n of them new, in a cache whose other slots are NaN."""

    def __init__(self, kv, n, heads, latent=512, block=64, seed=0, spare_rows=0, std=1.0):
        g = gen(seed)
        self.kv, self.n, self.heads, self.latent, self.block = list(kv), list(n), heads, latent, block
        B, width = len(kv), max([-(-k // block) for k in kv] + [1]) + 1
        used = sum(-(-k // block) for k in kv)
        pool = torch.randperm(used + 3, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.data = torch.full((used + 3, block, latent + 64), math.nan, dtype=torch.bfloat16, device="cuda")
        at = 0
        for b, k in enumerate(kv):
            m = -(-k // block)
            self.table[b, :m] = pool[at:at + m]
            rows = torch.full((m * block, latent + 64), math.nan, dtype=torch.bfloat16, device="cuda")
            rows[:k] = normal(g, k, latent + 64, std=std)
            self.data[pool[at:at + m].long()] = rows.view(m, block, latent + 64)
            at += m
        self.T = sum(n) + spare_rows
        q = normal(g, self.T, heads, latent + 64 + 8)
        self.ql, self.qr = q[..., :latent], q[..., latent:latent + 64]
        self.offsets = np.concatenate([[0], np.cumsum(n)]).tolist()
        self.scale = (latent + 64) ** -0.5

    def slot(self, b, j):
        return int(self.table[b, j // self.block]), j % self.block

    def run(self, causal=True, ws=None, scale=None, stream=None, lse=True):
        T, H = self.T, self.heads
        self.ws = torch.zeros(attn.moe_latent_attention_workspace_size(T, len(self.kv), H, self.latent), dtype=torch.uint8, device="cuda") if ws is None else ws
        out, l = Guarded((T, H, self.latent), torch.bfloat16), Guarded((T, H), torch.float32)
        attn.moe_latent_attention(self.ql, self.qr, attn.LatentCache(self.data), self.table, i32(self.offsets), i32(self.kv),
                                  self.scale if scale is None else scale, out.t, l.t if lse else None, self.ws, causal=causal, stream=stream)
        out.check(), l.check()
        return out.t, l.t

    def check(self, causal=True, scale=None):
        out, lse = self.run(causal, scale=scale)
        assert moe.moe_check_device_status(self.ws) == 0
        want, bound, want_lse, lse_bound = ref.latent_attention(self.ql, self.qr, self.data, self.table, self.offsets, self.kv,
                                                                float(np.float32(self.scale if scale is None else scale)), causal)
        end = self.offsets[-1]
        fill = torch.full_like(out[end:].view(torch.uint8), 0xA5)
        assert torch.equal(out[end:].view(torch.uint8), fill)                  # rows of no request
        nothing = torch.isinf(want_lse[:end])
        assert torch.equal(torch.isinf(lse[:end]), nothing)
        assert (out[:end][nothing] == 0).all()
        some = ~nothing
        within(out[:end][some], want[:end][some], bound[:end][some], "out")
        within(lse[:end][some], want_lse[:end][some], lse_bound[:end][some], "lse")
        return out, lse


LATENT = [  # kv, n, heads, latent, block
    ([1], [1], 1, 512, 64), ([1], [1], 16, 256, 16), ([2, 63, 64, 65], [1, 1, 1, 1], 16, 512, 16), ([127, 128, 129], [1, 2, 3], 8, 512, 128),
    ([1000], [1], 16, 512, 64), ([0, 5, 0, 300], [0, 1, 0, 2], 20, 512, 32), ([700, 1], [5, 1], 40, 256, 64), ([2500, 90, 4100], [1, 1, 1], 128, 512, 64),
    ([777], [3], 64, 512, 16), ([300, 65], [300, 65], 12, 512, 32), ([530], [130], 5, 256, 128), ([900, 17, 33], [4, 4, 4], 32, 512, 64),
    ([64] * 40, [1] * 40, 96, 512, 64), ([193, 450], [2, 1], 256, 256, 16), ([20000], [1], 16, 512, 64), ([3, 2, 1], [3, 2, 1], 3, 512, 16),
    ([5000, 6000, 100], [1, 4, 7], 17, 512, 128), ([257] * 3, [33] * 3, 2, 256, 32)]


@pytest.mark.parametrize("kv,n,heads,latent,block", LATENT)
@pytest.mark.parametrize("causal", [True, False])
def test_latent_attention_matches_the_definition(kv, n, heads, latent, block, causal):
    Step(kv, n, heads, latent, block, seed=sum(kv) + heads, spare_rows=2).check(causal)


def test_latent_attention_rows_that_see_nothing():
    """Requests without tokens in the cache, and new tokens before the first position."""
    for kv, n in (([0, 40], [3, 1]), ([2], [5]), ([0], [1])):
        Step(kv, n, 16, 512, 16, seed=1, spare_rows=1).check()


@pytest.mark.parametrize("B", [300, 2000, 8192])
def test_latent_attention_of_many_requests(B):
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 90, B)
    n = np.minimum(rng.integers(0, 3, B), kv)
    if B > 2000:
        n[rng.random(B) < 0.8] = 0
    Step(kv.tolist(), n.tolist(), 4, 256, 16, seed=B).check()


@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0, 2.0 ** 12, 1e30])
def test_latent_attention_scores_of_any_size(scale):
    """Weights from equal ones to a single one.  Past 2^24 of score a bound on the difference says nothing: there the largest wins alone."""
    s = Step([200, 900], [2, 1], 16, 512, 64, seed=2)
    if scale <= 1.0:
        s.check(scale=scale)
        return
    out, lse = s.run(scale=scale)
    assert moe.moe_check_device_status(s.ws) == 0
    q = torch.cat((s.ql, s.qr), -1).double()
    for b in range(2):
        k = s.data[s.table[b, : -(-s.kv[b] // 64)].long()].double().reshape(-1, 576)[:s.kv[b]]
        for t in range(s.offsets[b], s.offsets[b + 1]):
            seen = s.kv[b] - (s.offsets[b + 1] - t) + 1
            x = q[t] @ k[:seen].T
            top = x.topk(2).values
            sure = top[:, 0] - top[:, 1] > 1e-2           # two fp32 sums of this size differ by less
            assert sure.any()
            assert torch.equal(out[t][sure], k[x.argmax(-1)][sure][:, :512].to(torch.bfloat16))
            want = scale * top[:, 0]
            assert ((lse[t].double() - want).abs() <= 2.0 ** -12 * want.abs())[sure].all()


def test_latent_attention_scores_that_grow_along_the_cache():
    """Every tile outgrows the ones before it, by up to a hundred binades a tile."""
    for step in (3.0, 60.0):
        s = Step([640, 1500], [2, 1], 32, 512, 64, seed=3)
        s.ql, s.qr = torch.zeros_like(s.ql), torch.ones_like(s.qr)
        for b in range(2):
            for j in range(s.kv[b]):
                page, off = s.slot(b, j)
                s.data[page, off, 512:] = j / 64 * step / (64 * s.scale)
        s.check()


def test_latent_attention_does_not_meet_what_it_does_not_see():
    """NaN and infinities in slots past a request's end (in every Step) and in later tokens of the same request."""
    for bad in (math.nan, math.inf, -math.inf):
        s = Step([130, 640], [4, 3], 16, 512, 64, seed=4)
        clean, clean_lse = s.run()
        for b in range(2):
            page, off = s.slot(b, s.kv[b] - 1)             # the last token: seen by the last row alone
            s.data[page, off, 3] = bad
            s.data[page, off, 511] = bad
        out, lse = s.run()
        assert moe.moe_check_device_status(s.ws) == 0
        for b in range(2):
            lo, hi = s.offsets[b], s.offsets[b + 1]
            assert torch.equal(out[lo:hi - 1], clean[lo:hi - 1]) and torch.equal(lse[lo:hi - 1], clean_lse[lo:hi - 1])
            assert not torch.isfinite(out[hi - 1][:, [3, 511]].float()).any()
        assert torch.isfinite(clean.float()).all()


def test_latent_attention_nan_early_in_the_cache_reaches_every_row():
    for n in (1, 40):
        s = Step([900], [n], 16, 512, 64, seed=5)
        page, off = s.slot(0, 100)
        s.data[page, off, 17] = math.nan
        out, lse = s.run()
        assert out[:, :, 17].isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("what", ["descending", "past T", "negative kv", "long kv"])
def test_latent_attention_bad_lengths_are_reported_and_nothing_is_written(what):
    s = Step([100, 50], [2, 1], 16, 256, 16, seed=6)
    if what == "descending":
        s.offsets = [0, 2, 1]
    elif what == "past T":
        s.offsets = [0, 2, 4]
    elif what == "negative kv":
        s.kv = [100, -1]
    else:
        s.kv = [s.table.shape[1] * 16 + 1, 50]
    out, lse = s.run()
    assert moe.moe_check_device_status(s.ws) == moe.MOE_ERR_DEVICE_ASSERT
    assert (out.view(torch.uint8) == 0xA5).all() and (lse.view(torch.uint8) == 0xA5).all()


def test_latent_attention_bad_block_is_reported_and_read_as_block_0():
    s = Step([100], [1], 16, 256, 16, seed=7)
    s.data[0] = normal(gen(9), 16, 320)
    good = s.table.clone()
    for bad in (-1, s.data.shape[0], 2 ** 31 - 1):
        s.table = good.clone()
        s.table[0, 2] = 0
        want, _ = s.run()
        s.table[0, 2] = bad
        out, _ = s.run()
        assert moe.moe_check_device_status(s.ws) == moe.MOE_ERR_DEVICE_ASSERT
        assert torch.equal(out, want)
    s.table = good                                         # entries past the end are not read
    s.run()
    assert moe.moe_check_device_status(s.ws) == 0


def test_latent_attention_in_a_cache_of_more_than_2_to_the_31_values():
    block, latent = 128, 512
    nb = 2 ** 31 // (block * (latent + 64)) + 40
    data = torch.empty(nb, block, latent + 64, dtype=torch.bfloat16, device="cuda")
    g = gen(10)
    s = Step([700, 300], [1, 2], 16, latent, block, seed=11)
    small = s.data
    far = torch.arange(nb - small.shape[0], nb, device="cuda")
    data[far] = small
    s.data, s.table = data, torch.where(s.table >= 0, s.table + (nb - small.shape[0]), s.table)
    s.check()
    slot = torch.tensor([nb * block - 1, 5], device="cuda")
    c, k = normal(g, 2, latent), normal(g, 2, 64)
    attn.moe_latent_append(c, k, slot, attn.LatentCache(data), s.ws)
    assert torch.equal(data[nb - 1, block - 1], torch.cat((c, k), 1)[0]) and torch.equal(data[0, 5], torch.cat((c, k), 1)[1])


def test_latent_attention_is_the_same_again_and_without_lse():
    s = Step([3000, 40, 900], [1, 3, 40], 24, 512, 32, seed=12)
    out, lse = s.run()
    for _ in range(3):
        again, lse2 = s.run()
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    alone, _ = s.run(lse=False)
    assert torch.equal(alone, out)
    big = torch.full((1 << 27,), 0xFF, dtype=torch.uint8, device="cuda")       # a larger workspace that held other things
    moe.moe_workspace_init(big)
    again, lse2 = s.run(ws=big)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


# ------------------------------------------------- streams, graphs, a whole run

def test_calls_on_a_stream_of_their_own():
    s = Step([500, 20], [1, 2], 16, 512, 64, seed=13)
    out, _ = s.run()
    x, w = normal(gen(1), 5, 512), normal(gen(2), 512)
    y = torch.empty_like(x)
    attn.moe_rms_norm(x, w, 1e-6, y)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    other, y2 = s.run(stream=stream)[0], torch.empty_like(x)
    attn.moe_rms_norm(x, w, 1e-6, y2, stream=stream)
    stream.synchronize()
    assert torch.equal(other, out) and torch.equal(y2, y)


class Layer:
    """The operators one after another, as a layer with latent attention uses them, on buffers of T tokens of B requests."""

    def __init__(self, B, T, hidden=512, heads=16, latent=256, block=16, width=20, seed=0):
        g = gen(seed)
        self.heads, self.latent, self.block, self.T = heads, latent, block, T
        self.x, self.res = normal(g, T, hidden), normal(g, T, hidden)
        self.w_norm, self.w_latent = 1 + normal(g, hidden, std=0.1), 1 + normal(g, latent, std=0.1)
        wide = latent + 64
        self.w_q = attn.FP8Weight.from_dense(normal(g, heads * wide, hidden, std=hidden ** -0.5))
        self.w_kv = attn.FP8Weight.from_dense(normal(g, wide, hidden, std=hidden ** -0.5))
        self.cache = attn.LatentCache(torch.full((B * width, block, wide), math.nan, dtype=torch.bfloat16, device="cuda"))
        self.rope = attn.RotaryTable.make(64)
        self.ctx, self.new = i32([0] * B), i32([0] * B)
        self.free, self.head, self.next = torch.arange(B * width, dtype=torch.int32, device="cuda"), i32([0]), i32([0])
        self.table, self.kv, self.offsets = i32([[-1] * width] * B), i32([0] * B), i32([0] * (B + 1))
        self.slots, self.pos = torch.zeros(T, dtype=torch.int64, device="cuda"), i32([0] * T)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.h, self.y = torch.empty(T, hidden, **bf), torch.empty(T, hidden, **bf)
        self.q, self.ckv = torch.empty(T, heads * wide, **bf), torch.empty(T, wide, **bf)
        self.out = torch.zeros(T, heads, latent, **bf)
        self.lse = torch.zeros(T, heads, device="cuda")
        self.ws = attn.alloc_workspace(T, B, heads, self.cache, (self.w_q, self.w_kv))

    def step(self, ws=None):
        ws, T, H, L = self.ws if ws is None else ws, self.T, self.heads, self.latent
        attn.moe_kv_build_tables(self.ctx, self.new, self.block, self.free, self.head, self.table, self.kv, self.offsets, self.slots, self.pos, self.next, ws)
        attn.moe_rms_norm(self.x, self.w_norm, 1e-6, self.y, residual=self.res, residual_out=self.h)
        attn.moe_linear_fp8(self.y, self.w_q, self.q, ws)
        attn.moe_linear_fp8(self.y, self.w_kv, self.ckv, ws)
        q = self.q.view(T, H, L + 64)
        attn.moe_rotary(q[..., L:], self.pos, self.rope, q[..., L:])
        attn.moe_latent_append(self.ckv[:, :L], self.ckv[:, L:], self.slots, self.cache, ws, positions=self.pos, table=self.rope, norm=self.w_latent)
        attn.moe_latent_attention(q[..., :L], q[..., L:], self.cache, self.table, self.offsets, self.kv, (L + 64) ** -0.5, self.out, self.lse, ws)
        self.ctx.add_(self.new)
        self.head.copy_(self.next)


def check_layer(layer, before):
    """Each operator's output against its definition on what the one before it left."""
    L, H, n = layer.latent, layer.heads, int(layer.offsets[-1])
    want, bound, h, h_bound = ref.rms_norm(layer.x, float(np.float32(1e-6)), layer.w_norm, layer.res)
    within(layer.y, want, bound, "norm")
    within(layer.h, h, h_bound, "residual")
    plain = torch.empty_like(layer.q)
    attn.moe_linear_fp8(layer.y, layer.w_q, plain, layer.ws)
    pos, q = layer.pos[:n], layer.q.view(layer.T, H, L + 64)
    want, bound = ref.rotary(plain.view_as(q)[:n, :, L:], pos, layer.rope.turns)
    within(q[:n, :, L:], want, bound, "rotary")
    assert torch.equal(q[..., :L], plain.view_as(q)[..., :L])
    rows = layer.cache.data.view(-1, L + 64)[layer.slots[:n]]
    want, bound, _, _ = ref.rms_norm(layer.ckv[:n, :L], float(np.float32(1e-6)), layer.w_latent)
    within(rows[:, :L], want, bound, "latent")
    want, bound = ref.rotary(layer.ckv[:n, None, L:], pos, layer.rope.turns)
    within(rows[:, L:], want[:, 0], bound[:, 0], "key")
    kv = layer.kv.tolist()
    assert kv == [a + b for a, b in zip(before, layer.new.tolist())]
    want, bound, want_lse, lse_bound = ref.latent_attention(q[..., :L], q[..., L:], layer.cache.data, layer.table, layer.offsets.tolist(), kv,
                                                            float(np.float32((L + 64) ** -0.5)))
    within(layer.out[:n], want[:n], bound[:n], "attention")
    within(layer.lse[:n], want_lse[:n], lse_bound[:n], "lse")
    assert moe.moe_check_device_status(layer.ws) == 0


def test_the_operators_together_eager_and_captured():
    layer = Layer(B=3, T=12)
    layer.new.copy_(i32([5, 0, 7]))                        # prompts, one request without
    layer.step()
    check_layer(layer, [0, 0, 0])
    layer.new.copy_(i32([1, 3, 2]))
    ctx, head = layer.ctx.clone(), layer.head.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    assert torch.equal(layer.ctx, ctx) and torch.equal(layer.head, head)
    for new in ([1, 3, 2], [1, 1, 1], [12, 0, 0], [0, 0, 0], [0, 11, 1]):       # lengths on the device, other ones each time
        layer.new.copy_(i32(new))
        layer.x.mul_(-0.9)
        before = layer.ctx.tolist()
        graph.replay()
        check_layer(layer, before)


def test_two_captured_graphs_share_a_workspace():
    one, two = Step([900, 30], [1, 2], 64, 512, 64, seed=20), Step([2000], [3], 16, 512, 64, seed=21)
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    want = [s.run(ws=ws)[0].clone() for s in (one, two)]
    outs, graphs, keep = [], [], []
    for s in (one, two):
        out = torch.empty(s.T, s.heads, s.latent, dtype=torch.bfloat16, device="cuda")
        args = (attn.LatentCache(s.data), s.table, i32(s.offsets), i32(s.kv), s.scale, out, None, ws)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            attn.moe_latent_attention(s.ql, s.qr, *args)
        outs.append(out), graphs.append(g), keep.append(args)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert moe.moe_check_device_status(ws) == 0


# ------------------------------------------- the range-checked build, launch forms

def test_range_checked_build_finds_nothing_and_computes_the_same():
    steps = [Step([900, 30, 0, 4000], [1, 2, 0, 3], 64, 512, 64, seed=30), Step([3000], [1], 16, 256, 16, seed=31), Step([130, 700], [40, 9], 128, 512, 32, seed=32)]
    want = [s.run() for s in steps]
    with moe.debug_bounds():
        for s, (out, lse) in zip(steps, want):
            got, got_lse = s.run()
            assert moe.moe_check_device_status(s.ws) == 0
            assert torch.equal(got, out) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("kv,n,heads,plans", [([700] * 3, [1] * 3, 16, 0), ([64] * 152, [1] * 152, 64, 0), ([64] * 153, [1] * 153, 64, 1),
                                              ([9] * 300, [1] * 300, 8, 1), ([150], [150], 64, 0), ([2000], [2000], 16, 1), ([500] * 150, [1] * 150, 128, 0),
                                              ([70] * 100, [2] * 100, 40, 1)])
def test_latent_attention_on_both_sides_of_the_plan_kernel(kv, n, heads, plans, tmp_path):
    """Up to 152 units every CTA makes the plan itself, above a kernel before does."""
    s = Step(kv, n, heads, 512, 64, seed=len(kv))
    s.check()
    args = (attn.LatentCache(s.data), s.table, i32(s.offsets), i32(s.kv), s.scale, torch.empty_like(s.ql, memory_format=torch.contiguous_format), None, s.ws)
    names = [x for x in kernels(lambda: attn.moe_latent_attention(s.ql, s.qr, *args), tmp_path) if "latent" in x]
    assert has(names, "latent_plan_kernel") == bool(plans) and has(names, "latent_kernel", 512) and has(names, "latent_join_kernel", 512), names


@pytest.mark.parametrize("heads", [15, 16, 17, 47, 48, 49, 63, 64, 65, 80, 81, 96, 127, 128, 129, 160, 255, 256])
def test_latent_attention_head_counts_around_the_tiles(heads):
    """Units of 16 rows and of 64, two CTAs to a unit above, two units to a token above 128."""
    Step([200, 333, 64], [1, 1, 1], heads, 512, 64, seed=heads).check()
    Step([90, 130], [3, 2], heads, 256, 16, seed=heads).check()


@pytest.mark.parametrize("kv,n,heads", [([3000] * 8, [1, 2, 3, 4] * 2, 32), ([5000, 100, 4000], [1, 0, 1], 96), ([700] * 16, [1] * 16, 130),
                                        ([9000, 64], [2, 0], 80), ([2000, 65, 1], [1, 1, 1], 129), ([900] * 4, [1, 0, 0, 3], 100)])
def test_latent_attention_of_ragged_rows(kv, n, heads):
    """No more tokens than requests, and more: units that two CTAs share (a request's tokens may still be several), and units of 64 rows."""
    Step(kv, n, heads, 512, 64, seed=sum(n) + heads).check()
    Step(kv, n, heads, 256, 16, seed=sum(n) + heads).check(causal=False)


@pytest.mark.parametrize("kv,n", [([200], [1]), ([9000], [2]), ([700, 30], [3, 1])])
def test_latent_attention_scores_that_leave_fp32(kv, n):
    """Below: such tokens weigh nothing, the request's first one too; where all are, and above, the row is NaN."""
    s = Step(kv, n, 16, 512, 64, seed=40)
    s.ql, s.qr = torch.zeros_like(s.ql), torch.zeros_like(s.qr)
    s.ql[:, 0::2, 0] = 1e20                                # every second head: scores -1e40 of tokens with -1e20 there
    s.ql[..., 1] = 1.0
    for b in range(len(kv)):
        for j in range(kv[b]):
            page, off = s.slot(b, j)
            s.data[page, off, 0] = -1e20 if j % 3 == 0 else 0.0
    out, lse = s.run()
    assert moe.moe_check_device_status(s.ws) == 0
    for b in range(len(kv)):
        k = s.data[s.table[b, : -(-kv[b] // 64)].long()].double().reshape(-1, 576)[:kv[b]]
        for t in range(s.offsets[b], s.offsets[b + 1]):
            seen = kv[b] - (s.offsets[b + 1] - t) + 1
            x = (s.scale * k[:seen, 1]).clone()
            x[0::3] = -math.inf
            want, want_lse = torch.softmax(x, 0) @ k[:seen, 1:512], torch.logsumexp(x, 0)
            size = torch.softmax(x, 0) @ k[:seen, 1:512].abs()
            bound = (ref.U16 + 4 * seen * ref.U32) * size * (1 + ref.U16) + ref.U16 * want.abs() + 1e-30
            within(out[t, 0::2, 1:], want.expand(8, -1), bound.expand(8, -1))
            assert ((lse[t, 0::2].double() - want_lse).abs() < 1e-5).all()
    for value in (-1e20, 1e20):
        for b in range(len(kv)):
            for j in range(kv[b]):
                page, off = s.slot(b, j)
                s.data[page, off, 0] = value
        out, lse = s.run()
        assert out[:, 0::2, 1:].isnan().all() and lse[:, 0::2].isnan().all()
        assert torch.isfinite(out[:, 1::2, 1:].float()).all() and torch.isfinite(lse[:, 1::2]).all()


def test_latent_attention_rows_before_the_first_position_in_a_cut_unit():
    """A request with more new tokens than it has tokens at all, long enough for its units to be cut."""
    Step([900], [1400], 4, 256, 16, seed=41).check()
    Step([130], [135], 2, 512, 64, seed=42).check()


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own; what they share is the cache, which both read."""
    one, two = Step([20000, 300], [1, 2], 64, 512, 64, seed=50), Step([9000] * 5, [1] * 5, 96, 512, 16, seed=51)
    want = [s.run()[0] for s in (one, two)]
    outs = [torch.empty(s.T, s.heads, s.latent, dtype=torch.bfloat16, device="cuda") for s in (one, two)]
    args = [(attn.LatentCache(s.data), s.table, i32(s.offsets), i32(s.kv), s.scale, o, None, torch.zeros_like(s.ws)) for s, o in zip((one, two), outs)]
    x, w = normal(gen(3), 300, 2048), normal(gen(4), 2048)
    clean, y = torch.empty_like(x), torch.empty_like(x)
    attn.moe_rms_norm(x, w, 1e-6, clean)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a, stream in zip((one, two), args, streams):
            attn.moe_latent_attention(s.ql, s.qr, *a, stream=stream)
        attn.moe_rms_norm(x, w, 1e-6, y, stream=streams[2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, v) for o, v in zip(outs, want)) and torch.equal(y, clean)
    assert all(moe.moe_check_device_status(a[-1]) == 0 for a in args)


def test_right_behind_the_kernels_that_make_its_inputs():
    """Queries, lengths and cache written by the kernels just before, again and again: nothing is read early."""
    s = Step([700, 64, 1300], [1, 1, 1], 32, 512, 64, seed=52)
    source, lens = s.data.clone(), i32(s.kv)
    kv, ql, qr = torch.empty_like(lens), torch.empty(3, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 32, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    out = [torch.empty(3, 32, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    args = (attn.LatentCache(s.data), s.table, i32(s.offsets))
    weight, tokens = torch.ones(512, dtype=torch.bfloat16, device="cuda"), normal(gen(9), 3, 576)
    slots = torch.tensor([int(s.table[b, (k - 1) // 64]) * 64 + (k - 1) % 64 for b, k in enumerate(s.kv)], device="cuda")
    for i in range(30):
        for k in range(2):                                 # the second time with a wait in between: the same bits
            s.data.copy_(source)
            kv.copy_(lens)
            attn.moe_rms_norm(s.ql.reshape(96, 512) * (1 + i % 3), weight, 1e-6, ql.view(96, 512))
            attn.moe_rotary(s.qr.contiguous(), i32([i, 2, 3]), attn.RotaryTable.make(64), qr)
            attn.moe_latent_append(tokens[:, :512] * (1 + i % 5), tokens[:, 512:], slots, args[0], ws)
            if k:
                torch.cuda.synchronize()
            attn.moe_latent_attention(ql, qr, *args, kv, s.scale, out[k], None, ws)
        assert torch.equal(out[0], out[1]), i
    assert moe.moe_check_device_status(ws) == 0
