"""Attention of large scores: softmax references far from zero, ties, and scores past fp32, against the definition in 64 bits.

The queries and keys are chosen so that every score is exact in the kernels' arithmetic as well: a query is (A, A / 2^14, 0, ...), a
key 2^e (+-256, t, 0, ...) with whole t, and softmax_scale is log(2), which fp32's log2(e) turns into 1.  A score is then
A 2^e (+-256 + t / 2^14) to the base 2, and the only errors are those of the weights and of the result."""
import math

import numpy as np
import pytest
import torch

import attn_reference as ref
import test_gpu_attn as base

pytestmark = pytest.mark.gpu
built = base.built


def problem(lens, kv_heads, group, dim, size, k, sign, spread, seed, mixed=True):
    """Scores near sign * 2^k, apart by multiples of 2^(k - 22); in some blocks half as large (mixed)."""
    p = base.Problem(lens, kv_heads, group, dim, size, seed=seed)
    rng = np.random.default_rng(seed + 1)
    a = k // 2
    p.cache.k[:] = 0
    p.cache.k[..., 0] = ref.e4m3_codes(np.array(256.0 * sign))
    p.cache.k[..., 1] = ref.e4m3_codes(rng.integers(-spread, spread + 1, p.cache.k.shape[:3]).astype(np.float64))
    p.cache.ke[:] = k - a - 8
    if mixed:
        p.cache.ke -= rng.random(p.cache.ke.shape) < 0.3
    p.cache.ve[:] = rng.integers(-9, -4, p.cache.ve.shape)
    q = np.zeros(tuple(p.q.shape))
    q[..., 0], q[..., 1] = 2.0 ** a, 2.0 ** (a - 14)
    p.q = base.bf16(q)
    p.scale = math.log(2)
    return p


def units(p, causal=True, window=0):
    """For each request and query head: its rows of q, their scores to the base 2 (-infinity where a row does not see), the
    values, their exponents, the largest sum of a row's |terms|."""
    q = base.f64(p.q)
    for b, kv in enumerate(p.kv):
        lo, n = p.offsets[b], p.n[b]
        if n == 0 or kv == 0:
            continue
        pos, j = kv - n + np.arange(n)[:, None], np.arange(kv)[None]
        hide = (j > pos if causal else np.zeros((n, kv), bool)) | (j <= pos - window if window else False)
        for h in range(q.shape[1]):
            k, v, ve = p.cache.tokens(p.table[b], h // p.group, kv)
            x = np.where(hide, -np.inf, q[lo:lo + n, h] @ k.T)
            sees = ~hide.all(1)
            yield np.arange(lo, lo + n)[sees], h, x[sees], v, ve, (np.abs(q[lo:lo + n, h]) @ np.abs(k).T).max(1)[sees]


def check(p, causal=True, window=0):
    out, lse = p.run(causal, window)
    assert p.status == 0
    got, got_lse = base.f64(out), base.f64(lse)
    seen = np.zeros(got_lse.shape, bool)
    for t, h, x, v, ve, _ in units(p, causal, window):
        seen[t, h] = True
        m = x.max(1, keepdims=True)
        w = np.exp2(x - m)
        l = w.sum(1, keepdims=True)
        w /= l
        o = w @ v
        # f16 rounds a weight by 2^-11 of itself or 2^-25 of the largest weight x 2^exponent (times codes of at most 448); powers and
        # sums in fp32 by 2^-18; bf16 rounds the result by 2^-8
        bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -18) * (w @ np.abs(v)) + len(v) * 448 * 2.0 ** -25 * (w * 2.0 ** ve).max(1, keepdims=True)
        err = np.abs(got[t, h] - o)
        assert (err <= bound).all(), (t[0], h, float((err / bound).max()))
        want = (m + np.log2(l))[:, 0] * math.log(2)
        d = np.abs(got_lse[t, h] - want)
        assert (d <= 2.0 ** -15 + 2.0 ** -20 * np.abs(want)).all(), (t[0], h, float(d.max()))
    assert not got[~seen].any() and np.isneginf(got_lse[~seen]).all()


# requests, key/value heads, group, head size, block size of units of many rows: whole units, and cut ones beside them
MANY = {"64": ([(30, 300), (17, 140), (40, 40), (9, 3)], 8, 4, 64, 32), "128": ([(30, 300), (17, 140), (40, 40), (9, 3)], 8, 4, 128, 16),
        "64 cut": ([(8, 2000), (9, 700), (8, 400), (30, 130)], 8, 4, 64, 16), "128 cut": ([(8, 2000), (9, 700), (8, 400), (30, 130)], 8, 4, 128, 64),
        "128 two halves": ([(40, 900), (70, 300), (9, 100), (33, 64)], 8, 8, 128, 32), "64 two halves": ([(40, 900), (70, 300), (9, 100), (33, 64)], 8, 8, 64, 64)}
# units of up to 16, 32 and 64 rows, one that many CTAs share, and a plan that is made by a kernel before (more than 256 requests)
FEW = {"16 of 64": ([(1, 700), (2, 140), (4, 4), (1, 33), (3, 2)], 2, 4, 64, 32), "16 of 128": ([(1, 700), (2, 140), (4, 4), (1, 33), (3, 2)], 2, 4, 128, 16),
       "32 of 64": ([(3, 500), (4, 200), (3, 90)], 2, 8, 64, 64), "32 of 128": ([(3, 500), (4, 200), (3, 90)], 2, 8, 128, 16),
       "64 of 64": ([(8, 500), (5, 90)], 2, 8, 64, 32), "64 of 128": ([(8, 500), (5, 90)], 2, 8, 128, 128), "one of 64": ([(1, 9000)], 1, 2, 64, 32),
       "one of 128": ([(2, 7000)], 2, 8, 128, 64), "300 requests": ([(1, 1 + i % 140) for i in range(300)], 1, 2, 64, 16)}
FORMS = {**{f"many rows {k}": v for k, v in MANY.items()}, **{f"few rows {k}": v for k, v in FEW.items()}}


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("k", [0, 12, 18, 20, 21, 22, 24, 28, 32, 60, 120])
@pytest.mark.parametrize("form", FORMS)
def test_attention_scores_of_any_size(form, k, sign):
    lens, kv_heads, group, dim, size = FORMS[form]
    check(problem(lens, kv_heads, group, dim, size, k, sign, 16, seed=k))


@pytest.mark.parametrize("k", [10, 27, 40])
@pytest.mark.parametrize("form", FORMS)
def test_attention_equal_scores(form, k):
    """Every visible score is the same: the result is the values' mean, also where a unit's parts hold different numbers of tokens."""
    lens, kv_heads, group, dim, size = FORMS[form]
    p = problem(lens, kv_heads, group, dim, size, k, 1, 0, seed=k, mixed=False)
    check(p)
    check(p, causal=False, window=150)


@pytest.mark.parametrize("step", [1, 7, 25])
@pytest.mark.parametrize("form", FORMS)
def test_attention_scores_climb_past_fp32s_whole_numbers(form, step):
    """Keys' exponents climb from block to block, so that references move from ordinary scores to far ones inside tiles and units."""
    lens, kv_heads, group, dim, size = FORMS[form]
    for sign in (1, -1):
        p = problem(lens, kv_heads, group, dim, size, 12, sign, 16, seed=step, mixed=False)
        for row, kv in zip(p.table, p.kv):
            for i in range(-(-kv // size)):
                p.cache.ke[row[i]] = -2 + min(step * (i % 5), 90) * sign
        check(p)


@pytest.mark.parametrize("size", [2.0 ** 28, 2.0 ** 36])
@pytest.mark.parametrize("form", FORMS)
def test_attention_far_random_scores_pick_the_largest(form, size):
    """Random queries and keys with scores of this size: a row's largest score takes all the weight, wherever its lead is
    more than the sums' rounding."""
    lens, kv_heads, group, dim, size_ = FORMS[form]
    p = base.Problem(lens, kv_heads, group, dim, size_, seed=5, q_scale=size)
    p.scale = dim ** -0.5 * math.log(2)
    out, lse = p.run()
    got, got_lse = base.f64(out), base.f64(lse)
    assert p.status == 0
    clear = total = 0
    for t, h, x, v, _, terms in units(p):
        x, terms = x * dim ** -0.5, terms * dim ** -0.5
        top = np.sort(x, 1)[:, -2:]
        lead = top[:, 1] - top[:, 0] if x.shape[1] > 1 else np.full(len(x), np.inf)
        best = v[x.argmax(1)]
        assert (np.abs(got_lse[t, h] - top[:, -1] * math.log(2)) <= 2.0 ** -18 * terms).all() and np.isfinite(got[t, h]).all()
        sure = lead > 2.0 ** -18 * terms + 60
        assert (np.abs(got[t, h] - best)[sure] <= 2.0 ** -8 * np.abs(best[sure]) + 1e-30).all()
        clear, total = clear + sure.sum(), total + len(x)
    assert clear > 0.9 * total


@pytest.mark.parametrize("form", FORMS)
def test_attention_scores_past_fp32(form):
    """Where every score that a row sees is past fp32's range the row is NaN, not one that sees nothing; a score that is far below the
    range beside ordinary ones has no weight, as in the definition."""
    lens, kv_heads, group, dim, size = FORMS[form]
    for sign in (1, -1):
        p = problem(lens, kv_heads, group, dim, size, 120, sign, 16, seed=3, mixed=False)
        p.cache.ke += 20
        out, lse = p.run()
        assert p.status == 0
        seen = np.zeros(tuple(lse.shape), bool)
        for t, h, *_ in units(p):
            seen[t, h] = True
        o, ls = base.f64(out), base.f64(lse)
        assert np.isnan(o[seen]).all() and np.isnan(ls[seen]).all() and not o[~seen].any() and np.isneginf(ls[~seen]).all()
    p = problem(lens, kv_heads, group, dim, size, 12, -1, 16, seed=4, mixed=False)
    p.q = base.bf16(base.f64(p.q) * 2.0 ** 8)              # scores of -2^20, and of -2^148 in each request's first block
    first = [b for b, kv in enumerate(p.kv) if kv > size]
    p.cache.ke[p.table[first, 0]] = 126
    out, lse = p.run()
    assert p.status == 0
    got, got_lse = base.f64(out), base.f64(lse)
    for t, h, x, v, ve, _ in units(p):
        m = x.max(1, keepdims=True)
        w = np.exp2(x - m)
        l = w.sum(1, keepdims=True)
        ok = (m > -2.0 ** 100)[:, 0]                       # rows that see more than the first block
        o, want = (w / l) @ v, (m + np.log2(l))[:, 0] * math.log(2)
        bound = 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * ((w / l) @ np.abs(v)) + len(v) * 448 * 2.0 ** -25 * (w / l * 2.0 ** ve).max(1, keepdims=True)
        assert (np.abs(got[t, h] - o) <= bound)[ok].all() and (np.abs(got_lse[t, h] - want) <= 2.0 ** -20 * np.abs(want))[ok].all()
        assert np.isnan(got[t, h][~ok]).all()


@pytest.mark.parametrize("above", [12, 16, 20, 24])
@pytest.mark.parametrize("form", [f for f in FORMS if "300" not in f])
def test_attention_one_block_of_far_larger_values_leaves_the_others_their_bits(form, above):
    """A visible block with an exponent far above the others', and values in the first half of the dims only: the other half is made of the
    other blocks, whose weights are small beside that block's contribution."""
    lens, kv_heads, group, dim, size = FORMS[form]
    p = base.Problem(lens, kv_heads, group, dim, size, seed=6, exps=(-7, -7), q_scale=0.3)
    for b, kv in enumerate(p.kv):
        block = p.table[b, (kv - p.n[b]) // size // 2]     # seen by every row
        p.cache.ve[block] = -7 + above
        p.cache.v[block, :, :, dim // 2:] = 0
    out, _ = p.run()
    assert p.status == 0
    got, half = base.f64(out), dim // 2
    for t, h, x, v, ve, _ in units(p):
        x = x * p.scale * math.log2(math.e)
        w = np.exp2(x - x.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        o, top = w @ v, (w * 2.0 ** ve).max(1, keepdims=True)
        # a weight (times 2^exponent) is off by 2^-11 of itself or up to 2^-30 of the row's largest, evenly: 2^-30.8 in the mean square, times
        # codes of 90 in the mean square (448 x 2^-2.3); six times that, summed over the row, is below half of the last term;
        # scores in fp32 by less than 2^-14
        bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13) * (w @ np.abs(v)) + 6 * math.sqrt(len(v)) * 2.0 ** -32 * top * 448
        err = np.abs(got[t, h] - o)[:, half:]
        assert (err <= bound[:, half:] + 1e-30).all(), (t[0], h, float((err / (bound[:, half:] + 1e-30)).max()))
