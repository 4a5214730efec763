"""A decoder layer served in 8 bits: the layer's quantized products, the norm that
feeds them, the key/value cache and the attention over it, as they run together.

    layer = Int8DecoderLayer(norm1, qkv, out, norm2, up, down, heads, kv_heads)
    cache = new_cache(n_pages, n_slots, kv_heads, head_dim)
    y, r = layer(x, None, cache, page_table, lengths, cu, max_q=..., max_len=...)  # prompts
    y, r = layer(x, None, cache, page_table, lengths)                              # one token each

Pre-norm: r = x + residual, a = out(attention(qkv(norm1(r)))), r' = r + a,
y = down(gelu(up(norm2(r')))); the caller passes (y, r') on to the next layer,
whose norm adds them.  All four products are LLM.int8() layers, which set the
outlier columns of their rows apart ([blog, "A closer look at the MatMul"]); the
norms then give 16-bit rows.  ``codes=True`` takes the norm's row codes for qkv and
up instead (rmsnorm_quant -> linear_codes: one pass over the rows and no 16-bit
copy of them).  A row of codes has one scale: a column of 60 among unit values
makes its steps 0.47, an error of 14 % of each unit value where rows without
outlier columns have about 1 %.  That path is for models whose normed rows have
none; it takes 0.58 ms instead of 0.80 for a prompt of 2048 rows, 0.16 instead of
0.27 for 16 single tokens (hidden 4096, 32 heads of 128 on 8, 16384 features in
between).  Positions enter as linear biases (``alibi``) or not at all.  What has no
kernel in the library, the norm to 16 bits and the activation function, is torch's.
"""
from __future__ import annotations

import torch

from . import quantize_weight as _quantize_weight
from .module import Int8Linear
from .serving import _inference, cache_attention, cache_write, linear_codes, rmsnorm_quant


class _CodesLinear(torch.nn.Module):
    """y = codes . W^T + b for row codes (Xq, sx): the weight of an nn.Linear as
    codes, no fp16 copy and no outlier columns."""

    def __init__(self, lin: torch.nn.Linear, device):
        super().__init__()
        with torch.no_grad():
            W = lin.weight.detach().to(device, torch.float16).t().contiguous()   # [in][out]
            Wq, sw = _quantize_weight(W)
            b = None if lin.bias is None else lin.bias.detach().to(device, torch.float16)
        self.register_buffer("Wq", Wq)
        self.register_buffer("sw", sw)
        self.register_buffer("bias", b)

    def forward(self, Xq, sx):
        return linear_codes(Xq, sx, self.Wq, self.sw, bias=self.bias)


class Int8DecoderLayer(torch.nn.Module):
    """One pre-norm decoder layer over packed rows x fp16 [rows][hidden] (inference).

    ``threshold``: from which magnitude on a column of a product's rows is an outlier
    column.  ``has_fp16_weights``: the products keep their weights in 16 bits too, for the
    rows of outlier columns (False: those rows are rebuilt from the codes, which saves two
    bytes a weight; a code's rounding, about 1 % of a feature's weights, is then
    multiplied by the outlier).  ``codes``: qkv and up on the norm's row codes, with no
    outlier columns."""

    def __init__(self, norm1, qkv, out, norm2, up, down, heads, kv_heads=None, alibi=None,
                 eps=1e-5, threshold=6.0, device="cuda", codes=False,
                 has_fp16_weights=True):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        hidden = qkv.in_features
        if heads % kv_heads or qkv.out_features % (heads + 2 * kv_heads):
            raise ValueError(f"qkv has {qkv.out_features} features for {heads} query and "
                             f"{kv_heads} kv heads")
        self.heads, self.kv_heads = heads, kv_heads
        self.head_dim = qkv.out_features // (heads + 2 * kv_heads)
        if out.in_features != heads * self.head_dim or out.out_features != hidden or \
                up.in_features != hidden or down.in_features != up.out_features or \
                down.out_features != hidden:
            raise ValueError("out, up and down must fit qkv's sizes")
        self.eps, self.codes = eps, bool(codes)
        self.register_buffer("norm1", norm1.detach().to(device, torch.float16))
        self.register_buffer("norm2", norm2.detach().to(device, torch.float16))
        def product(lin):
            return Int8Linear.from_linear(lin, has_fp16_weights=has_fp16_weights, threshold=threshold,
                                          device=device).requires_grad_(False)

        self.qkv, self.up = ((_CodesLinear(qkv, device), _CodesLinear(up, device)) if codes else
                             (product(qkv), product(up)))
        self.out, self.down = product(out), product(down)
        self.register_buffer("alibi", None if alibi is None else
                             torch.as_tensor(alibi, dtype=torch.float32).to(device))

    def _norm_product(self, lin, x, residual, weight):
        """(lin(norm of r), r), r = x + residual."""
        if self.codes:
            Xq, sx, r = rmsnorm_quant(x, weight, residual=residual, eps=self.eps)
            return lin(Xq, sx), r
        r = x if residual is None else x + residual
        h = r.float()
        rms = torch.sqrt(h.square().mean(dim=1, keepdim=True) + self.eps)
        return lin((h / rms * weight.float()).half()), r

    def forward(self, x, residual, cache, page_table, lengths, cu=None, slots=None, max_q=None,
                max_len=None, window=0):
        """(y, r') of rows x (+ residual): the last rows of their sequences, whose keys
        and values the call appends to ``cache``; page_table, lengths (this call's rows
        included), cu, slots, max_q and max_len as for ``cache_attention``."""
        _inference(x, residual)
        with torch.no_grad():
            rows, D, H = x.shape[0], self.head_dim, self.heads
            qkv, r = self._norm_product(self.qkv, x, residual, self.norm1)
            qkv = qkv.view(rows, H + 2 * self.kv_heads, D)
            q, k, v = qkv[:, :H], qkv[:, H:H + self.kv_heads], qkv[:, H + self.kv_heads:]
            cache_write(cache, k, v, page_table, lengths, cu=cu, slots=slots, max_new=max_q)
            a = cache_attention(q, cache, page_table, lengths, cu=cu, slots=slots, max_q=max_q,
                                max_len=max_len, window=window, alibi=self.alibi)
            up, r = self._norm_product(self.up, self.out(a.view(rows, H * D)), r, self.norm2)
            return self.down(torch.nn.functional.gelu(up)), r
