"""Float64 oracle of the operators around the attention: per-head norm and rotation, the paged cache, attention of
drafted tokens over it.  Plain loops and definitions on CPU tensors; float64 throughout.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def rotate(x, cos, sin, interleaved, inverse=False):
    """x [..., d] turned by cos, sin [..., rope/2]."""
    r = 2 * cos.shape[-1]
    sin = -sin if inverse else sin
    out = x.clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def _angles(cos, sin, positions, B, N):
    """Each row's cos and sin [B,1,N,rope/2], and which rows are padding [B,1,N,1]."""
    pos = torch.arange(N).expand(B, N) if positions is None else positions.long()
    if cos is None:
        e = torch.zeros(B, 1, N, 0, dtype=F64)
        return e, e, torch.zeros(B, 1, N, 1, dtype=torch.bool)
    at = pos.clamp(0, cos.shape[0] - 1)
    c, s = cos.to(F64)[at], sin.to(F64)[at]
    far = (pos >= cos.shape[0])[..., None]
    return (torch.where(far, math.nan, c)[:, None], torch.where(far, math.nan, s)[:, None],
            (pos < 0)[:, None, :, None])


def norm_rope(x, w, cos, sin, positions, eps, interleaved):
    """(rotated, normed before the rotation) of x [B,H,N,d]."""
    x = x.to(F64)
    B, _, N, d = x.shape
    c, s, pad = _angles(cos, sin, positions, B, N)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.to(F64)
    return torch.where(pad, 0.0, rotate(y, c, s, interleaved)), torch.where(pad, 0.0, y)


def norm_rope_grad(x, dz, w, cos, sin, positions, eps, interleaved):
    """dx, dw and the magnitudes that bound their rounding errors: r (|g| + |xh| mean |g xh|), sum |dy xh|."""
    x, dz = x.to(F64), dz.to(F64)
    B, _, N, d = x.shape
    c, s, pad = _angles(cos, sin, positions, B, N)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dy = rotate(dz, c, s, interleaved, inverse=True)
    xh = x * r
    g = dy if w is None else dy * w.to(F64)
    dx = torch.where(pad, 0.0, r * (g - xh * (g * xh).mean(-1, keepdim=True)))
    terms = torch.where(pad, 0.0, dy * xh)
    mag = r * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    return dx, terms.sum((0, 1, 2)), torch.where(pad, 0.0, mag), terms.abs().sum((0, 1, 2))


def e4m3_row(x):
    """(values, exponent byte) of one row [d] quantised to e4m3 with a power-of-two scale; magnitudes stop at
    1.875 * 2^127, so that every value is a bf16 number."""
    x = x.to(F64)
    if not torch.isfinite(x).all():
        return torch.full_like(x, math.nan), 255
    x = x.clamp(-1.875 * 2.0 ** 127, 1.875 * 2.0 ** 127)
    top = float(x.abs().max())
    k = -100
    while top > 448.0 * 2.0 ** k:
        k += 1
    y = x / 2.0 ** k
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp_min(-6) - 3)
    return torch.round(y / step) * step * 2.0 ** k, k + 127


def row_place(table, lens, n_new, T, page_size, pages, b, t):
    """(page, slot) of new token t of sequence b, or None."""
    nn = T if n_new is None else min(max(int(n_new[b]), 0), T)
    j = max(int(lens[b]), 0) - nn + t
    if t >= nn or not 0 <= j < table.shape[1] * page_size:
        return None
    p = int(table[b, j // page_size])
    return (p, j % page_size) if 0 <= p < pages else None


def sequence(values, table, length, page_size, b):
    """Rows 0..length-1 of sequence b from values [pages, Hk, page_size, d], [Hk, length, d] and which exist."""
    pages, hk, _, d = values.shape
    out = torch.zeros(hk, length, d, dtype=F64)
    there = torch.zeros(length, dtype=torch.bool)
    for j in range(min(length, table.shape[1] * page_size)):
        p = int(table[b, j // page_size])
        if 0 <= p < pages:
            out[:, j] = values[p, :, j % page_size]
            there[j] = True
    return out, there


def tree_attention(q, kvals, vvals, table, lens, n_new, tree, scale):
    """O, L and two magnitudes per row (sum of p |v| [.., d], largest sum of |q k| scale) of drafted tokens; kvals and
    vvals are the cache's values [pages, Hk, page_size, d] in float64, tree a list of Python ints per sequence and
    token (bit j: token j is seen) or None."""
    B, H, T, d = q.shape
    pages, hk, ps, _ = kvals.shape
    o = torch.zeros(B, H, T, d, dtype=F64)
    lse = torch.full((B, H, T), -math.inf, dtype=F64)
    mag = torch.zeros(B, H, T, d, dtype=F64)
    dot = torch.zeros(B, H, T, dtype=F64)
    cap = table.shape[1] * ps
    for b in range(B):
        nn = T if n_new is None else min(max(int(n_new[b]), 0), T)
        prefix = max(int(lens[b]), 0) - nn
        n = min(max(int(lens[b]), 0), cap)
        k, there = sequence(kvals, table, n, ps, b)
        v, _ = sequence(vvals, table, n, ps, b)
        for t in range(nn):
            see = there.clone()
            for j in range(max(prefix, 0), n):
                dj = j - prefix
                see[j] &= dj <= t if tree is None else bool(tree[b][t] >> dj & 1)
            idx = see.nonzero()[:, 0]
            if len(idx) == 0:
                continue
            for h in range(H):
                g = h // (H // hk)
                prod = q[b, h, t].to(F64) * k[g, idx]
                s = prod.sum(-1) * scale
                w = torch.softmax(s, 0)
                o[b, h, t] = w @ v[g, idx]
                lse[b, h, t] = torch.logsumexp(s, 0)
                mag[b, h, t] = w @ v[g, idx].abs()
                dot[b, h, t] = prod.abs().sum(-1).max() * scale
    return o, lse, mag, dot
