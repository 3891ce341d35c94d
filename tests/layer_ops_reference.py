"""Norm, rotary positions, latent append and latent attention from their definitions, in 64 bits, for the tests.
Shares no code with the package.  Each comes with the bound of the kernels' error, from their arithmetic:
bf16 rounds by at most 2^-8 of a value, fp32 by 2^-24."""
from __future__ import annotations

import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def unit(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def rms_norm(x, eps, weight=None, residual=None, post=None, gate=None, scale=1.0, wide=False):
    """(y, bound, h, bound).  fp32: a row's sum of squares passes fewer than 64 additions in a row (32 of a thread's values, 10 of the join), so
    that the norm's factor is within 40 units of 2^-24 (half of the sum's 64, root, quotient and product); products and the sum of h add fewer than 8."""
    u = x.double()
    if post is not None:
        u = unit(u, eps) * post.double()
    if gate is not None:
        u = u * gate.double()
    u = scale * u
    r = torch.zeros_like(u) if residual is None else residual.double()
    h = r + u
    slack = 48 * U32 * (u.abs() + r.abs())
    h_bound = slack + (0 if wide else U16 * h.abs()) + 1e-38
    if weight is None:
        return None, None, h, h_bound
    w = weight.double()
    y = unit(h, eps) * w
    # an error of h moves y by itself over the root mean square, and by its share of the mean
    rms = torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    moved = (slack + h.abs() * (slack * h.abs()).mean(-1, keepdim=True) / rms ** 2) / rms * w.abs()
    return y, U16 * y.abs() + 48 * U32 * y.abs() + 1.01 * moved + 1e-38, h, h_bound


def angles(positions, turns):
    """p f modulo one turn, exactly, in radians: [tokens, pairs]."""
    rows = []
    for p in positions.tolist():
        rows.append([((p * (t % (1 << 64))) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for t in turns.tolist()])
    return torch.tensor(rows, dtype=torch.float64).reshape(len(rows), turns.numel())


def rotary(x, positions, turns, amplitude=1.0, interleaved=False, offset=0, norm=None, eps=1e-6):
    """(values, bound) of x [tokens, heads, dim].  The angle is within 2^-25 turns (its rounding to fp32) and cosine and sine within 2 units of
    their last places: 2^-22 of the pair's size; the products and the sum add 3 units, a norm 48."""
    v = x.double()
    loss = 8 * U32 + 2 * math.pi * 2.0 ** -25
    if norm is not None:
        v = unit(v, eps) * norm.double()
        loss += 48 * U32
    t = angles(positions, turns).to(v.device)[:, None]
    part = 2 * turns.numel()
    cos, sin = torch.cos(t), torch.sin(t)
    p = v[..., offset:offset + part]
    a, b = (p[..., 0::2], p[..., 1::2]) if interleaved else (p[..., :part // 2], p[..., part // 2:])
    ra, rb = amplitude * (a * cos - b * sin), amplitude * (b * cos + a * sin)
    size = abs(amplitude) * (a.abs() + b.abs())

    def join(first, second):
        return torch.stack((first, second), -1).flatten(-2) if interleaved else torch.cat((first, second), -1)
    out, bound = v.clone(), loss * v.abs()
    out[..., offset:offset + part] = join(ra, rb)
    bound[..., offset:offset + part] = loss * join(size, size)
    return out, bound + U16 * out.abs() + 1e-38


def latent_attention(ql, qr, data, table, q_offsets, kv_lens, scale, causal=True):
    """out, bound of out, lse, bound of lse [T, heads, ...]; rows of no request are NaN in all four.
    A product q.k is exact, its fp32 sum over W terms within W 2^-24 of the sum of magnitudes (however it is ordered), so that a score is within
    delta; a weight is within 2 delta + 8 units (difference, exponential) of 2^-24 and, rounded to bf16, 2^-8 of itself; sums of n weights within
    n 2^-24 of theirs."""
    T, H, L = ql.shape
    out = torch.full((T, H, L), math.nan, dtype=torch.float64, device=ql.device)
    lse = torch.full((T, H), math.nan, dtype=torch.float64, device=ql.device)
    out_bound, lse_bound = out.clone(), lse.clone()
    block = data.shape[1]
    q = torch.cat((ql, qr), -1).double()
    for b, kv in enumerate(kv_lens):
        lo, hi = q_offsets[b], q_offsets[b + 1]
        if hi == lo:
            continue
        pages = table[b, : -(-kv // block)].long()
        k = data[pages].double().reshape(-1, L + 64)[:kv]
        for t in range(lo, hi):
            seen = max(0, min(kv, kv - (hi - t) + 1)) if causal else kv
            if seen == 0:
                out[t], lse[t], out_bound[t], lse_bound[t] = 0, -math.inf, 0, 0
                continue
            x = scale * (q[t] @ k[:seen].T)
            delta = (scale * (L + 64) * U32 * (q[t].abs() @ k[:seen].abs().T)).amax(-1) + 4 * U32 * x.abs().amax(-1)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - m)
            l = p.sum(-1, keepdim=True)
            o = (p @ k[:seen, :L]) / l
            size = (p @ k[:seen, :L].abs()) / l
            loss = (2 * torch.expm1(2 * delta) + (16 + 2 * seen) * U32)[:, None]
            out[t], lse[t] = o, (m + torch.log(l))[:, 0]
            out_bound[t] = (U16 + loss) * size * (1 + U16) + U16 * o.abs() + 1e-38
            lse_bound[t] = 2 * delta + (8 + seen) * U32 + 4 * U32 * lse[t].abs()
    return out, out_bound, lse, lse_bound
