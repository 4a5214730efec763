"""A decoder layer served in 8 bits: the layer's quantized products, the norm that
feeds them, the key/value cache and the attention over it, as they run together.

    layer = Int8DecoderLayer(norm1, qkv, out, norm2, up, down, heads, kv_heads)
    cache = new_cache(n_pages, n_slots, kv_heads, head_dim)
    y, r = layer(x, None, cache, page_table, lengths, cu, max_q=..., max_len=...)  # prompts
    y, r = layer(x, None, cache, page_table, lengths)                              # one token each
    # trees of drafted tokens (tree_plan), then the accepted ones (tree_accept) into the cache
    y, r, kv = layer.draft(x, None, cache, page_table, lengths, positions, masks, cu)
    layer.accept(kv, cache, page_table, new_lengths, path, counts, cu)

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
between).  Positions enter as linear biases (``alibi``), by rotation of queries and keys
(``rotary``; with norms of their heads, if given), or not at all.  What has no
kernel in the library, the norm to 16 bits and the activation function, is torch's.
"""
from __future__ import annotations

import torch

from . import quantize_weight as _quantize_weight
from .module import Int8Linear
from .positions import cache_append, rotate_heads, tree_attention
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
    outlier columns.  ``rotary``: a ``Rotary`` for queries and keys; ``q_norm`` and ``k_norm``
    [head_dim]: the weights of their heads' norms (eps ``head_eps``)."""

    def __init__(self, norm1, qkv, out, norm2, up, down, heads, kv_heads=None, alibi=None,
                 eps=1e-5, threshold=6.0, device="cuda", codes=False,
                 has_fp16_weights=True, rotary=None, q_norm=None, k_norm=None, head_eps=1e-6):
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
        self.rotary, self.head_eps = rotary, head_eps
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            self.register_buffer(name, None if w is None else w.detach().to(device, torch.float16))
        self._turned = any(x is not None for x in (rotary, q_norm, k_norm))

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
            q, k, v, r = self._heads(x, residual)
            if self._turned:
                q = cache_append(cache, k, v, page_table, lengths, q=q, rotary=self.rotary,
                                 q_weight=self.q_norm, k_weight=self.k_norm, eps=self.head_eps, cu=cu,
                                 slots=slots, max_new=max_q, q_out=q)
            else:
                cache_write(cache, k, v, page_table, lengths, cu=cu, slots=slots, max_new=max_q)
            a = cache_attention(q, cache, page_table, lengths, cu=cu, slots=slots, max_q=max_q,
                                max_len=max_len, window=window, alibi=self.alibi, out=self._answers(q, cu))
            return self._rest(a, r)

    def draft(self, x, residual, cache, page_table, lengths, positions, masks, cu=None, slots=None,
              max_q=None, max_len=None, window=0):
        """(y, r', kv) of rows x (+ residual) that are drafted tokens, trees of them behind
        their sequences: lengths counts the cached tokens alone, positions and masks are
        ``tree_plan``'s, the rest as for ``tree_attention``.  The cache is left as it is;
        kv, the rows' keys and values, is for ``accept``."""
        _inference(x, residual)
        with torch.no_grad():
            q, k, v, r = self._heads(x, residual)
            if self._turned:
                q, k = rotate_heads(q, positions, self.rotary, k=k, q_weight=self.q_norm,
                                    k_weight=self.k_norm, eps=self.head_eps, q_out=q, k_out=k)
            a = tree_attention(q, k, v, cache, page_table, lengths, masks, positions=positions, cu=cu,
                               slots=slots, max_q=max_q, max_len=max_len, window=window,
                               alibi=self.alibi, out=self._answers(q, cu))
            return (*self._rest(a, r), (k, v))

    def accept(self, kv, cache, page_table, lengths, path, counts, cu=None, slots=None, max_new=None):
        """Appends the accepted drafts among kv to the cache: path, counts and lengths (the
        new ones) as ``tree_accept`` gives them."""
        cache_append(cache, *kv, page_table, lengths, cu=cu, slots=slots, max_new=max_new,
                     counts=counts, index=path)

    def _heads(self, x, residual):
        """(q, k, v, r): heads of the rows, before norm and rotation."""
        D, H = self.head_dim, self.heads
        qkv, r = self._norm_product(self.qkv, x, residual, self.norm1)
        qkv = qkv.view(x.shape[0], H + 2 * self.kv_heads, D)
        return qkv[:, :H], qkv[:, H:H + self.kv_heads], qkv[:, H + self.kv_heads:], r

    def _answers(self, q, cu):
        """Where attention writes.  With cu there may be rows that it leaves as they are; the
        next product's outlier columns are those of all of its rows, so these hold 0 (a
        launch: 3 us of 145 or 209 for 16 x 8 rows, with and without ``codes``, 4 of 575 or
        745 for 2048, 10 of 1780 or 2220 for 8192; sizes as above)."""
        return None if cu is None else q.new_zeros(q.shape)

    def _rest(self, a, r):
        """(y, r') from the attention's output on."""
        a = self.out(a.view(a.shape[0], self.heads * self.head_dim))
        up, r = self._norm_product(self.up, a, r, self.norm2)
        return self.down(torch.nn.functional.gelu(up)), r
