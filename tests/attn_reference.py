"""The attention half from its definitions, in 64 bits on the CPU, for the
tests: the 8-bit format, the cache layout, the tables, the append, the attention and
the block-scaled projection.  Shares no code with the package."""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------- the 8-bit format

def e4m3_table() -> np.ndarray:
    """The value of each E4M3 code (OCP: bias 7, no infinities, S.1111.111 is NaN)."""
    out = np.zeros(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[code] = np.nan if code & 0x7F == 0x7F else (-v if code & 0x80 else v)
    return out


TABLE = e4m3_table()
_POSITIVE = TABLE[:127]                                # ascending, 0 .. 448


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """Nearest code of each value (|v| <= 448), ties to the even code; 0x7F for what is not finite."""
    v = np.asarray(v, dtype=np.float64)
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == _POSITIVE[hi], hi, code)
    return np.where(np.isfinite(v), code | np.where(np.signbit(v), 128, 0), 127).astype(np.uint8)


def least_exponent(a: float) -> int:
    """The smallest e >= -126 with a <= 448 * 2^e."""
    e = -126
    while a > 448 * 2.0 ** e:
        e += 1
    return e


def finite_max(v: np.ndarray) -> float:
    v = np.abs(v[np.isfinite(v)])
    return float(v.max()) if v.size else 0.0


def quantise_groups(x: np.ndarray, size: int = 128):
    """Rows in groups along the last axis: (codes, exponents)."""
    rows, k = x.shape
    codes, exps = np.zeros((rows, k), np.uint8), np.zeros((rows, -(-k // size)), np.int64)
    for g in range(exps.shape[1]):
        cols = slice(g * size, min(k, (g + 1) * size))
        for r in range(rows):
            exps[r, g] = least_exponent(finite_max(x[r, cols]))
            codes[r, cols] = e4m3_codes(x[r, cols] / 2.0 ** exps[r, g])
    return codes, exps


# --------------------------------------------------------------- the cache

class Cache:
    """Codes as [block, head, token, dim] and exponents as [block, head]."""

    def __init__(self, blocks, heads, dim, block_size):
        self.size = block_size
        self.k, self.v = (np.zeros((blocks, heads, block_size, dim), np.uint8) for _ in range(2))
        self.ke, self.ve = (np.zeros((blocks, heads), np.int64) for _ in range(2))

    @staticmethod
    def from_layout(k, v, ks, vs):
        nb, heads, subs, chunks = k.shape[:4]
        c = Cache(nb, heads, 16 * chunks, 16 * subs)
        c.k = k.transpose(0, 1, 2, 4, 3, 5).reshape(nb, heads, 16 * subs, 16 * chunks).copy()
        c.v = v.transpose(0, 1, 2, 4, 3).reshape(nb, heads, 16 * subs, 16 * chunks).copy()
        c.ke, c.ve = ks.astype(np.int64) - 127, vs.astype(np.int64) - 127
        return c

    def layout(self):
        nb, heads, size, dim = self.k.shape
        k = self.k.reshape(nb, heads, size // 16, 16, dim // 16, 16).transpose(0, 1, 2, 4, 3, 5)
        v = self.v.reshape(nb, heads, size // 16, 16, dim).transpose(0, 1, 2, 4, 3)
        return (np.ascontiguousarray(k), np.ascontiguousarray(v), (self.ke + 127).astype(np.uint8), (self.ve + 127).astype(np.uint8))

    def append(self, k, v, slots):
        """k, v [T, heads, dim] doubles, slots [T] in runs of consecutive offsets of one block."""
        t = 0
        while t < len(slots):
            if slots[t] < 0:
                t += 1
                continue
            block, first = divmod(int(slots[t]), self.size)
            n = 1
            while t + n < len(slots) and slots[t + n] == slots[t] + n and int(slots[t + n]) // self.size == block:
                n += 1
            for x, codes, exps in ((k, self.k, self.ke), (v, self.v, self.ve)):
                for h in range(x.shape[1]):
                    e = least_exponent(finite_max(x[t:t + n, h]))
                    if first > 0:
                        old = exps[block, h]
                        if e > old:
                            codes[block, h, :first] = e4m3_codes(TABLE[codes[block, h, :first]] * 2.0 ** float(old - e))
                        e = max(e, old)
                    exps[block, h] = e
                    codes[block, h, first:first + n] = e4m3_codes(x[t:t + n, h] / 2.0 ** float(e))
            t += n

    def tokens(self, pages, head, n):
        """(keys, values, value exponents) of the first n tokens behind a table row."""
        pages = np.asarray(pages[: -(-n // self.size)], dtype=np.int64)
        k = TABLE[self.k[pages, head]] * 2.0 ** self.ke[pages, head][:, None, None]
        v = TABLE[self.v[pages, head]] * 2.0 ** self.ve[pages, head][:, None, None]
        d = k.shape[-1]
        return k.reshape(-1, d)[:n], v.reshape(-1, d)[:n], np.repeat(self.ve[pages, head], self.size)[:n]


# -------------------------------------------------------------- the tables

def build_tables(ctx, new, size, free, head, table, t_max):
    table = table.copy()
    slots, positions = np.full(t_max, -1, np.int64), np.full(t_max, -1, np.int64)
    offsets, t = [0], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        for i in range(-(-c // size), -(-(c + n) // size)):
            table[b, i] = free[head]
            head += 1
        for p in range(c, c + n):
            slots[t], positions[t] = int(table[b, p // size]) * size + p % size, p
            t += 1
        offsets.append(t)
    return table, [c + n for c, n in zip(ctx, new)], offsets, slots, positions, head


# ----------------------------------------------------------- the attention

def attention(q, cache: Cache, table, q_offsets, kv_lens, scale, causal=True, window=0):
    """out, lse and the bound on |out - exact| of a kernel that rounds the
    softmax weights to f16 (relative to the row's largest contribution) and the
    result to bf16, with fp32 sums: see bound below."""
    T, heads, d = q.shape
    group = heads // cache.k.shape[1]
    out, lse, bound = np.zeros((T, heads, d)), np.full((T, heads), -np.inf), np.zeros((T, heads, d))
    for b, kv in enumerate(kv_lens):
        lo, hi = q_offsets[b], q_offsets[b + 1]
        n = hi - lo
        for h in range(heads):
            if n == 0:
                continue
            k, v, ve = cache.tokens(table[b], h // group, kv)
            for i in range(n):
                p = kv - n + i
                first = max(0, p - window + 1) if window else 0
                last = min(kv, p + 1) if causal else kv
                if first >= last:
                    continue
                x = scale * (k[first:last] @ q[lo + i, h])
                m = x.max()
                w = np.exp(x - m)
                l = w.sum()
                lse[lo + i, h] = m + np.log(l)
                vv = v[first:last]
                o = (w / l) @ vv
                out[lo + i, h] = o
                # |x| <= s: a score is off by at most d * 2^-22 of its terms' sum s (fp32 products' sums, one
                # multiplication, 2^x in fp32), so weights by 2 * that; f16 rounds a weight by 2^-11 of itself or by
                # 2^-25 of the largest weight x 2^exponent, times codes of at most 448; bf16 by 2^-8 of the result
                s = scale * (np.abs(k[first:last]) @ np.abs(q[lo + i, h])).max()
                top = (w / l * 2.0 ** ve[first:last]).max()
                bound[lo + i, h] = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -18 + 2 * s * d * 2.0 ** -22) * ((w / l) @ np.abs(vv)) +
                                    (last - first) * 448 * 2.0 ** -25 * top)
    return out, lse, bound


# ---------------------------------------------------------- the projection

def linear(x, codes, scale_bytes):
    """y = X^ W^T in doubles, and the bound of fp32 sums over K (in K / 32
    steps, each off by at most 2^-22 of the terms' sum) and one rounding to bf16."""
    k = x.shape[1]
    xc, xe = quantise_groups(x)
    xq = TABLE[xc] * 2.0 ** np.repeat(xe, 128, axis=1)[:, :k].astype(np.float64)
    s = np.repeat(np.repeat(scale_bytes.astype(np.float64) - 127, 128, axis=0)[: codes.shape[0]], 128, axis=1)[:, :k]
    w = TABLE[codes] * 2.0 ** s
    y = xq @ w.T
    return y, 2.0 ** -8 * np.abs(y) + (k / 32 + 8) * 2.0 ** -22 * (np.abs(xq) @ np.abs(w).T)
