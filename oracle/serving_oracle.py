"""CPU oracle of the serving operators: plain torch on the CPU, float64 except
for the quantization decisions, which the method takes in IEEE float32 (a code
is an integer decided by floating point).  Test infrastructure only.

Every function follows the formulas of include/int8lin.h ("Serving in 8 bits
around the layer") with loops over sequences and heads; the HIP path shares no
code with it.
"""
from __future__ import annotations

import math

import torch

F32, F64 = torch.float32, torch.float64
LEAST = 2.0 ** -93   # an absmax below this counts as 0


def codes(x, absmax):
    """clamp(round_half_away(fl32(x) * fl32(127 / absmax)), -127, 127); 0 where absmax is 0."""
    x, absmax = x.to(F32), absmax.to(F32)
    inv = torch.where(absmax > 0, torch.tensor(127.0, dtype=F32) / absmax, torch.zeros_like(absmax))
    p = (x * inv).to(F64)           # the float32 product, then exact arithmetic
    r = torch.sign(p) * torch.floor(p.abs() + 0.5)
    return r.clamp(-127, 127).to(torch.int8)


def rmsnorm_quant(X, weight=None, residual=None, eps=1e-5):
    """(Xq int8, sx float64, h): h in X's type."""
    h = X if residual is None else (X.to(F32) + residual.to(F32)).to(X.dtype)
    g = h.to(F32) if weight is None else h.to(F32) * weight.to(F32)
    top = g.abs().amax(dim=1, keepdim=True)
    top = torch.where(top < LEAST, torch.zeros_like(top), top)
    rms = torch.sqrt(h.to(F64).square().mean(dim=1) + eps)
    sx = top[:, 0].to(F64) / rms
    return codes(g, top), torch.where(top[:, 0] == 0, torch.zeros_like(sx), sx), h


def linear_codes(Xq, sx, Wq, sw, bias=None):
    """(Y float64, the magnitude sum |product| + |bias|)."""
    acc = Xq.to(F64) @ Wq.to(F64).t()
    p = acc * sx.to(F64)[:, None] * sw.to(F64) / (127.0 * 127.0)
    b = torch.zeros_like(p) if bias is None else bias.to(F64).expand_as(p)
    return p + b, p.abs() + b.abs()


class Store:
    """What a cache should hold: the 16-bit tokens of each sequence, and from them
    the codes and scales of every complete page."""

    def __init__(self, page_size):
        self.P = page_size

    def page(self, x):
        """(codes [P][D], scale float32) of one page of one head, x [P][D]."""
        top = x.abs().to(F32).max() if torch.isfinite(x.to(F32)).all() else torch.tensor(math.inf)
        if not math.isfinite(float(top)):
            return torch.zeros(x.shape, dtype=torch.int8), torch.tensor(math.nan, dtype=F32)
        top = torch.where(top < LEAST, torch.zeros_like(top), top)
        return codes(x, top), top / torch.tensor(127.0, dtype=F32)

    def sequence(self, x):
        """float32 values [n][H][D] that the cache stands for, x [n][H][D] 16-bit; and
        per page and head its codes and scale."""
        n, H, D = x.shape
        val, pages = x.to(F32).clone(), []
        for g in range(n // self.P):
            rows = slice(g * self.P, (g + 1) * self.P)
            per = [self.page(x[rows, h]) for h in range(H)]
            pages.append(per)
            for h, (c, s) in enumerate(per):
                val[rows, h] = c.to(F32) * s
        return val, pages


def attention(q, k, v, scale, window=0, alibi=None, page_scale=None, u=2.0 ** -11):
    """One sequence: q [m][Hq][D] (the queries of its last m tokens), k, v [n][H][D] the
    cache's values.  Returns (out float64 [m][Hq][D], tolerance of the same shape).

    The tolerance bounds what fp32 scores and sums and 16-bit weights can do, from
    the values at hand (u: unit roundoff of the 16-bit type):
      - a score is a sum of D products in fp32 with a few roundings after it, so it
        errs by at most (D + 8) 2^-24 times its magnitude sum, and the weights by
        that factor (twice: numerator and denominator);
      - weights are rounded to 16 bits once (u, of sum p |v|; an fp16 weight below
        2^-14 by 2^-25 of the largest contribution), sums of n terms in fp32 err by
        n 2^-24, the result is rounded once (u).
    page_scale [n][H]: the scale that a code of token t stands for (1 in the tail)."""
    m, Hq, D = q.shape
    n, H, _ = k.shape
    G = Hq // H
    out = torch.zeros((m, Hq, D), dtype=F64)
    tol = torch.zeros_like(out)
    if n == 0:
        return out, tol
    back = torch.arange(n - m, n)[:, None] - torch.arange(n)[None]      # [m][n]
    seen = back >= 0
    if window:
        seen &= back < window
    count = seen.sum(1, keepdim=True).to(F64)
    some = count[:, 0] > 0
    for h in range(Hq):
        kk, vv, qq = k[:, h // G].to(F64), v[:, h // G].to(F64), q[:, h].to(F64)
        s = qq @ kk.T * scale
        mag = qq.abs() @ kk.abs().T * abs(scale)
        if alibi is not None:
            bias = float(alibi[h]) * back.to(F64)
            s, mag = s - bias, mag + bias.abs()
        p = torch.softmax(s.masked_fill(~seen, -math.inf), dim=1)
        p = torch.where(some[:, None], p, torch.zeros_like(p))
        o = p @ vv
        es = (D + 8) * 2.0 ** -24 * (torch.where(seen, mag, torch.zeros_like(mag)) + 64.0).amax(1, keepdim=True)
        e = 2 * es + 2 * (count + 64) * 2.0 ** -24
        out[:, h] = o
        tol[:, h] = (u + e) * (p @ vv.abs()) + u * o.abs() + 2.0 ** -24
        if u < 2.0 ** -8:   # fp16: the weights' subnormal range
            sv = torch.ones(n, dtype=F64) if page_scale is None else page_scale[:, h // G].to(F64)
            c = vv.abs() / torch.where(sv > 0, sv, torch.ones_like(sv))[:, None]
            tol[:, h] += 2.0 ** -25 * (p * sv).amax(1, keepdim=True) * (seen.to(F64) @ c)
    return out, torch.where(some[:, None, None], tol, torch.zeros_like(tol))
