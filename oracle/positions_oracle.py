"""CPU oracle of rotary positions and of drafted tokens over the cache: plain torch on
the CPU in float64.  Test infrastructure only.

Every function follows the formulas of include/int8lin.h ("Positions, and drafted
tokens over the cache") with loops over rows, pairs and drafts where that is the plainest
way; the HIP path shares no code with it.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def unit(dtype):
    """Half a step of the type, relative."""
    return torch.finfo(dtype).eps / 2


def pairs(n, interleaved):
    """(first, second) element of each of n pairs."""
    i = torch.arange(n)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + n)


def turn(x, positions, freqs, interleaved, factor=1.0):
    """x float64 [rows][heads][D] turned to its rows' positions."""
    a, b = pairs(freqs.numel(), interleaved)
    t = positions.to(F64)[:, None, None] * freqs.to(F64)
    y = x.clone()
    y[..., a] = factor * (x[..., a] * torch.cos(t) - x[..., b] * torch.sin(t))
    y[..., b] = factor * (x[..., a] * torch.sin(t) + x[..., b] * torch.cos(t))
    return y


def norm(x, weight, eps):
    if weight is None:
        return x
    rms = torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return torch.where(rms > 0, x / torch.where(rms > 0, rms, 1.0), 0.0) * weight


def spread(mag, positions, freqs, interleaved, factor):
    """What an element is made of: for a pair factor (|a| + |b|) on both, else |x|."""
    a, b = pairs(freqs.numel(), interleaved)
    out = mag.clone()
    out[..., a] = out[..., b] = abs(factor) * (mag[..., a] + mag[..., b])
    return out


def rotate(x, positions, freqs, interleaved=False, factor=1.0, weight=None, eps=1e-6):
    """(y float64, tolerance) of x [rows][heads][D] in a 16-bit type.

    The tolerance: one rounding to the type; before it, in fp32, at most 24 roundings of
    2^-24 in the norm (a sum of 16 squares and 4 partial sums, halved by the root, root,
    quotient, three products), 8 in an angle's sine and cosine (a turn's fraction is within
    2^-25, 3.2 of them after the factor 2 pi, the functions within 1.3e-7, 2.2 of them, the
    factor one), 3 in the pair's products and sum: below 2^-19 of what the element is made
    of.  Past 2^20 turns the angle is formed in 64 bits: 3 roundings of 2^-53 of its size
    (below, its fraction in two 32-bit parts is within the 2^-25 above)."""
    d = x.to(F64)
    w = None if weight is None else weight.to(F64)
    n = norm(d, w, eps)
    y = turn(n, positions, freqs, interleaved, factor)
    size = 2.0 ** -19 + 2.0 ** -51 * (positions.to(F64).abs().max() * max([*freqs.abs().tolist(), 0.0])
                                      if positions.numel() else 0.0)
    tiny = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps   # half a subnormal step, twice
    return y, unit(x.dtype) * y.abs() + size * spread(n.abs(), positions, freqs, interleaved, factor) + tiny


def rotate_grad(dy, x, positions, freqs, interleaved=False, factor=1.0, weight=None, eps=1e-6):
    """((dx, tolerance), (dweight, tolerance) or None) in float64, by the formula.

    Tolerances: g errs by 2^-19 of what it is made of, as in the forward pass, the normed
    x by 2^-19 of itself, the mean of their D products by that of both and 24 roundings
    more: dx by less than 2^-16 of the magnitudes that it is formed from.  The sum of a
    weight's gradient has below 128 additions on a path."""
    g = turn(dy.to(F64), -positions, freqs, interleaved, factor)
    G = spread(dy.to(F64).abs(), positions, freqs, interleaved, factor)
    u, tiny = unit(dy.dtype), torch.finfo(dy.dtype).smallest_normal * torch.finfo(dy.dtype).eps
    if weight is None:
        return (g, u * g.abs() + 2.0 ** -19 * G + tiny), None
    d, w = x.to(F64), weight.to(F64)
    rms = torch.sqrt(d.square().mean(-1, keepdim=True) + eps)
    r = torch.where(rms > 0, 1.0 / torch.where(rms > 0, rms, 1.0), 0.0)
    n = d * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    made = r * (G * w.abs() + n.abs() * (G * w.abs() * n.abs()).mean(-1, keepdim=True))
    dw, dw_made = (g * n).sum((0, 1)), (G * n.abs()).sum((0, 1))
    return ((dx, u * dx.abs() + 2.0 ** -16 * made + tiny),
            (dw, u * dw.abs() + 2.0 ** -16 * dw_made + tiny))


def tree_plan(parents, length):
    """(positions, masks as lists of sets) of one sequence's drafts."""
    positions, seen = [], []
    for j, p in enumerate(parents):
        own = 0 <= p < j
        seen.append({j} | (seen[p] if own else set()))
        positions.append(length + len(seen[j]) - 1)
    return positions, seen


def words(seen, n_words):
    """Sets of drafts as int64 [rows][n_words]."""
    out = torch.zeros((len(seen), n_words), dtype=torch.int64)
    for j, s in enumerate(seen):
        for i in s:
            bit = 1 << (i & 63)
            out[j, i >> 6] |= bit - (1 << 64) if bit >> 63 else bit
    return out


def tree_accept(parents, tokens, choices, first=None):
    """(accepted drafts in order, the token chosen to follow them) of one sequence."""
    n = len(parents)
    own = [p if 0 <= p < j else -1 for j, p in enumerate(parents)]
    if first is None:
        if not n:
            return [], -1
        path, want = [0], choices[0]
    else:
        path, want = [], first
    while True:
        cur = path[-1] if path else -1
        for j in range(n):
            if own[j] == cur and tokens[j] == want and (path or own[j] == -1):
                path.append(j)
                want = choices[j]
                break
        else:
            return path, want


def tree_attention(q, k, v, scale, seen, back=None, slopes=None, page_scale=None, dtype=torch.float16):
    """One sequence: q [m][Hq][D]; k, v [n][H][D], the cache's values and then the drafts;
    seen [m][n]; back [m][n] the distance of each key, with slopes [Hq].  Returns (out
    float64, tolerance).

    The tolerance: a score is a sum of D products in fp32 with a few roundings after it,
    so it errs by at most (D + 8) 2^-24 of its magnitude sum (64 for the exponential's own
    range), and the weights by that factor, twice; they are rounded to 16 bits once (u of
    sum p |v|; an fp16 weight below 2^-14 by 2^-25 of the largest contribution, where the
    contribution of a coded key counts its page_scale [n][H], 1 for the others); sums of n
    terms in fp32 err by n 2^-24, the result is rounded once."""
    m, Hq, D = q.shape
    n, H, _ = k.shape
    u = unit(dtype)
    out = torch.zeros((m, Hq, D), dtype=F64)
    tol = torch.zeros_like(out)
    if n == 0 or m == 0:
        return out, tol
    count = seen.sum(1, keepdim=True).to(F64)
    some = count[:, 0] > 0
    for h in range(Hq):
        kv = h // (Hq // H)
        kk, vv, qq = k[:, kv].to(F64), v[:, kv].to(F64), q[:, h].to(F64)
        s, mag = qq @ kk.T * scale, qq.abs() @ kk.abs().T * abs(scale)
        if slopes is not None:
            bias = float(slopes[h]) * back.to(F64)
            s, mag = s - bias, mag + bias.abs()
        p = torch.softmax(s.masked_fill(~seen, -math.inf), dim=1)
        p = torch.where(some[:, None], p, 0.0)
        es = (D + 8) * 2.0 ** -24 * (torch.where(seen, mag, 0.0) + 64.0).amax(1, keepdim=True)
        e = 2 * es + 2 * (count + 64) * 2.0 ** -24
        out[:, h] = p @ vv
        tol[:, h] = (u + e) * (p @ vv.abs()) + u * out[:, h].abs() + 2.0 ** -24
        if dtype == torch.float16:
            sv = torch.ones(n, dtype=F64) if page_scale is None else page_scale[:, kv].to(F64)
            c = vv.abs() / torch.where(sv > 0, sv, 1.0)[:, None]
            tol[:, h] += 2.0 ** -25 * (p * sv).amax(1, keepdim=True) * (seen.to(F64) @ c)
    return out, torch.where(some[:, None, None], tol, 0.0)
