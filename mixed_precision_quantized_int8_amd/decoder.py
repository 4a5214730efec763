"""A decoder layer served in 8 bits: the layer's quantized products, the norm that
feeds them, the key/value cache and the attention over it, as they run together.

    layer = Int8DecoderLayer(norm1, qkv, out, norm2, up, down, heads, kv_heads)
    cache = new_cache(n_pages, n_slots, kv_heads, head_dim)
    y, r = layer(x, None, cache, page_table, lengths, cu, max_q=..., max_len=...)  # prompts
    y, r = layer(x, None, cache, page_table, lengths)                              # one token each

Pre-norm: r = x + residual, a = out(attention(qkv(norm1(r)))), r' = r + a,
y = down(gelu(up(norm2(r')))); the caller passes (y, r') on to the next layer,
whose norm adds them.  qkv and up take the norm's row codes (rmsnorm_quant ->
linear_codes); out and down take fp16 rows and keep the layer's outlier
decomposition ([blog, "A closer look at the MatMul"]).  Positions enter as linear
biases (``alibi``) or not at all.  Everything runs in the library's kernels but
the activation function.
"""
from __future__ import annotations

import torch

from . import quantize_weight as _quantize_weight
from .module import Int8Linear
from .serving import cache_attention, cache_write, linear_codes, rmsnorm_quant


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
    """One pre-norm decoder layer over packed rows x fp16 [rows][hidden] (inference)."""

    def __init__(self, norm1, qkv, out, norm2, up, down, heads, kv_heads=None, alibi=None,
                 eps=1e-5, threshold=6.0, device="cuda"):
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
        self.eps = eps
        self.register_buffer("norm1", norm1.detach().to(device, torch.float16))
        self.register_buffer("norm2", norm2.detach().to(device, torch.float16))
        self.qkv, self.up = _CodesLinear(qkv, device), _CodesLinear(up, device)
        self.out = Int8Linear.from_linear(out, threshold=threshold, device=device)
        self.down = Int8Linear.from_linear(down, threshold=threshold, device=device)
        self.register_buffer("alibi", None if alibi is None else
                             torch.as_tensor(alibi, dtype=torch.float32).to(device))

    @torch.no_grad()
    def forward(self, x, residual, cache, page_table, lengths, cu=None, slots=None, max_q=None,
                max_len=None, window=0):
        """(y, r') of rows x (+ residual): the last rows of their sequences, whose keys
        and values the call appends to ``cache``; page_table, lengths (this call's rows
        included), cu, slots, max_q and max_len as for ``cache_attention``."""
        Xq, sx, r = rmsnorm_quant(x, self.norm1, residual=residual, eps=self.eps)
        rows, D, H = x.shape[0], self.head_dim, self.heads
        qkv = self.qkv(Xq, sx).view(rows, H + 2 * self.kv_heads, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + self.kv_heads], qkv[:, H + self.kv_heads:]
        cache_write(cache, k, v, page_table, lengths, cu=cu, slots=slots, max_new=max_q)
        a = cache_attention(q, cache, page_table, lengths, cu=cu, slots=slots, max_q=max_q,
                            max_len=max_len, window=window, alibi=self.alibi)
        Xq, sx, r = rmsnorm_quant(self.out(a.view(rows, H * D)), self.norm2, residual=r,
                                  eps=self.eps)
        return self.down(torch.nn.functional.gelu(self.up(Xq, sx))), r
