"""Serving in 8 bits around the layer: the norm that feeds a product with row
codes, the product of codes that are already there, a key/value cache held in 8
bits, and attention over it.  Marshalling only, as in the package's __init__:
every step runs in the HIP kernels of libint8lin.so (include/int8lin.h states
the formulas).  For inference: there are no gradients, and a tensor that requires
one is refused where torch records them.

    Xq, sx, h = rmsnorm_quant(X, weight, residual=r)   # norm of X + r as row codes
    Y = linear_codes(Xq, sx, Wq, sw)                   # their product with a weight
    cache = new_cache(n_pages, n_slots, heads, head_dim)
    cache_write(cache, k, v, page_table, lengths)      # one new token per sequence
    o = cache_attention(q, cache, page_table, lengths) # and its attention
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _binding
from ._binding import check, lib

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_byref = ctypes.byref


def _on(device):
    """Makes ``device`` the current one for a call (nothing to do if it is)."""
    return contextlib.nullcontext() if device.index == torch.cuda.current_device() \
        else torch.cuda.device(device)


# the handle of torch's current stream (through the Stream object where this torch has
# no direct way: 2 us of a call whose kernel takes 3)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _inference(*tensors):
    """Refuses tensors that would need a gradient: these operators have none, and a result
    without one would end the graph unnoticed."""
    for t in tensors:
        if getattr(t, "requires_grad", False) and torch.is_grad_enabled():
            raise RuntimeError("the serving operators have no gradients, but an argument requires "
                               "one: call them under torch.no_grad() or detach it")


def _dense(t, dtype, shape, device, name):
    """The pointer of a contiguous tensor of this type, shape and device (None: any
    GPU); these calls are short, so what is right is settled first, what is wrong
    said after."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and \
            t.is_contiguous() and (t.is_cuda if device is None else t.device == device):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'a GPU'} (got {t.device})")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _result(t, dtype, shape, device, name):
    """(tensor, pointer) to write a result to: the caller's, or a new one."""
    if t is not None:
        return t, _dense(t, dtype, shape, device, name)
    t = torch.empty(shape, dtype=dtype, device=device)
    return t, t.data_ptr()


def _scratch(workspace, nbytes, device):
    """(pointer, bytes) of the caller's workspace, or of a new one; the tensor lives
    until its memory may be given to later work of the same stream."""
    if workspace is None:
        if not nbytes:
            return None, None, 0
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    n = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
    return workspace, _dense(workspace, torch.uint8, (n,), device, "workspace"), n


def _half_type(t, name, dims):
    """The dtype code of a GPU tensor in fp16 or bf16 with this many dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16 or bfloat16 (got {t.dtype})")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(t.shape)}")
    return code


def rmsnorm_quant(X, weight=None, residual=None, eps=1e-5, Xq=None, sx=None, residual_out=None):
    """Residual addition, root-mean-square norm and int8 row codes.

    X [M][K] fp16 or bf16 (residual, weight [K] and residual_out of its type) ->
    (Xq int8 [M][K], sx fp32 [M], h [M][K]): h = X + residual rounded to the
    type (X itself without a residual), Xq * sx / 127 the norm of h times
    ``weight`` (None: ones), one scale per row.  Statistics in fp32.  ``Xq``,
    ``sx`` and ``residual_out`` (which may be ``residual`` or ``X``) receive the
    results if given.  No outlier columns are set apart: a column c times as large
    as the others leaves those 127 / c steps (``linear`` on 16-bit rows has them).
    """
    _inference(X, weight, residual)
    code = _half_type(X, "X", 2)
    (M, K), dev, dt = X.shape, X.device, X.dtype
    x = _dense(X, dt, (M, K), None, "X")
    w = None if weight is None else _dense(weight, dt, (K,), dev, "weight")
    r = None if residual is None else _dense(residual, dt, (M, K), dev, "residual")
    Xq, qp = _result(Xq, torch.int8, (M, K), dev, "Xq")
    sx, sp = _result(sx, torch.float32, (M,), dev, "sx")
    h, hp = X, None
    if residual_out is not None or residual is not None:
        h, hp = _result(residual_out, dt, (M, K), dev, "residual_out")
    with _on(dev):
        check(lib().int8_rmsnorm_quant(x, r, w, M, K, float(eps), code, qp, sp, hp, _stream(dev)))
    return Xq, sx, h


def linear_codes(Xq, sx, Wq, sw, bias=None, out=None, workspace=None):
    """Product of row codes with a quantized weight, no outlier columns:
    Y = fp16(acc * sx * sw / 127^2 + bias) with acc = Xq . Wq^T exact in int32.

    Xq int8 [M][K] with sx fp32 [M] (``rmsnorm_quant``), Wq int8 [N][K] with sw
    fp32 [N] (``quantize_weight``), bias fp16 [N] -> Y fp16 [M][N].  ``workspace``
    (uint8) takes the partial sums of shapes that are split along K (for more than
    64 rows); None allocates what the shape needs.
    """
    _inference(sx, sw, bias)
    if not isinstance(Xq, torch.Tensor) or not isinstance(Wq, torch.Tensor):
        raise TypeError("Xq and Wq must be torch.Tensors")
    if Xq.dim() != 2 or Wq.dim() != 2:
        raise ValueError(f"Xq and Wq must be matrices, got {list(Xq.shape)} and {list(Wq.shape)}")
    (M, K), N, dev = Xq.shape, Wq.shape[0], Xq.device
    xp = _dense(Xq, torch.int8, (M, K), None, "Xq")
    wp = _dense(Wq, torch.int8, (N, K), dev, "Wq")
    b = None if bias is None else _dense(bias, torch.float16, (N,), dev, "bias")
    out, op = _result(out, torch.float16, (M, N), dev, "out")
    need = 0 if workspace is not None or M <= 64 else int(lib().i8l_codes_workspace_bytes(M, K, N))
    hold, ws, nb = _scratch(workspace, need, dev)
    with _on(dev):
        check(lib().int8_linear_codes(
            xp, _dense(sx, torch.float32, (M,), dev, "sx"), M, K, wp,
            _dense(sw, torch.float32, (N,), dev, "sw"), N, b, op, ws, nb, _stream(dev)))
    return out


class KVCache:
    """A key/value cache in 8 bits, in pages of P tokens with one scale for each
    page and kv head, over tensors that the caller owns:

      k_codes int8 [n_pages][heads][P][head_dim]   value = code * scale
      v_codes int8 [n_pages][heads][head_dim][P]
      k_scale, v_scale fp32 [n_pages][heads]
      k_tail [n_slots][heads][P][head_dim], v_tail [n_slots][heads][head_dim][P]
          fp16 or bf16: the tokens of each sequence's last, incomplete page

    P is 16, 32, 64 or 128; head_dim a multiple of 16 up to 256.  The cache holds the
    tensors' addresses: its attributes do not change (a larger pool is a new KVCache over
    new tensors), and the tensors must not be resized or given other storage.
    """

    __slots__ = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "heads",
                 "page_size", "head_dim", "dtype", "device", "_struct")

    def __init__(self, k_codes, v_codes, k_scale, v_scale, k_tail, v_tail):
        code = _half_type(k_tail, "k_tail", 4)
        if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4:
            raise ValueError("k_codes must be a tensor [n_pages][heads][page_size][head_dim]")
        n, H, P, D = k_codes.shape
        slots, dev, dt = k_tail.shape[0], k_codes.device, k_tail.dtype
        struct = _binding.KVCacheStruct(
            _dense(k_codes, torch.int8, (n, H, P, D), None, "k_codes"),
            _dense(v_codes, torch.int8, (n, H, D, P), dev, "v_codes"),
            _dense(k_scale, torch.float32, (n, H), dev, "k_scale"),
            _dense(v_scale, torch.float32, (n, H), dev, "v_scale"),
            _dense(k_tail, dt, (slots, H, P, D), dev, "k_tail"),
            _dense(v_tail, dt, (slots, H, D, P), dev, "v_tail"), n, slots, H, D, P, code)
        for put, x in zip(_CACHE_FIELDS, (k_codes, v_codes, k_scale, v_scale, k_tail, v_tail, H, P, D,
                                          dt, dev, struct)):
            put(self, x)

    def __setattr__(self, name, x):
        raise AttributeError(f"{name}: a KVCache does not change; make a new one over new tensors")

    def __delattr__(self, name):
        raise AttributeError(f"{name}: a KVCache does not change")

    @property
    def n_pages(self):
        return self._struct.n_pages

    @property
    def n_slots(self):
        return self._struct.n_slots


# what the constructor writes an unchanging cache's attributes with
_CACHE_FIELDS = [KVCache.__dict__[name].__set__ for name in KVCache.__slots__]


def new_cache(n_pages, n_slots, heads, head_dim, page_size=64, dtype=torch.float16,
              device="cuda"):
    """A ``KVCache`` over new tensors (their contents do not matter: a token is
    read only after it has been written)."""
    def empty(shape, dt):
        return torch.empty(shape, dtype=dt, device=device)

    return KVCache(empty((n_pages, heads, page_size, head_dim), torch.int8),
                   empty((n_pages, heads, head_dim, page_size), torch.int8),
                   empty((n_pages, heads), torch.float32), empty((n_pages, heads), torch.float32),
                   empty((n_slots, heads, page_size, head_dim), dtype),
                   empty((n_slots, heads, head_dim, page_size), dtype))


def _sequences(cache, page_table, lengths, cu, slots):
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 tensor [sequences][pages]")
    (n, most), dev = page_table.shape, cache.device
    return _binding.SequencesStruct(
        _dense(page_table, torch.int32, (n, most), dev, "page_table"),
        _dense(lengths, torch.int32, (n,), dev, "lengths"),
        None if cu is None else _dense(cu, torch.int32, (n + 1,), dev, "cu"),
        None if slots is None else _dense(slots, torch.int32, (n,), dev, "slots"), n, most)


def _rows(t, cache, heads, name):
    """(pointer, token stride, head stride) of a [rows][heads][head_dim] tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != cache.dtype:
        raise TypeError(f"{name} must be {cache.dtype} (got {t.dtype})")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device} (got {t.device})")
    if t.dim() != 3 or t.shape[2] != cache.head_dim or (heads and t.shape[1] != heads):
        raise ValueError(f"{name} must be [rows][{heads or 'heads'}][{cache.head_dim}], "
                         f"got {list(t.shape)}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr(), st, sh


def _one_each(t, n, cu, name):
    if cu is None and t.shape[0] != n:
        raise ValueError(f"{name} must have one row for each of the {n} sequences (or pass cu), "
                         f"got {t.shape[0]}")


def cache_write(cache, k, v, page_table, lengths, cu=None, slots=None, max_new=None):
    """Appends keys and values to the sequences of a cache.

    k, v [rows][heads][head_dim] of the cache's type (strided views are fine:
    multiples of 8 elements).  Sequence i's rows are cu[i] .. cu[i+1] - 1 (int32
    [n+1]; None: row i alone) and become its last tokens: ``lengths`` (int32 [n])
    counts them in.  ``page_table`` int32 [n][pages] names its pages (tokens past them
    are skipped), ``slots`` int32 [n] its tail slot (None: slot i).  ``max_new``: at least the rows of any
    one sequence (None: all rows; a closer bound launches fewer workgroups).
    """
    _inference(k, v)
    s = _sequences(cache, page_table, lengths, cu, slots)
    kp, kt, kh = _rows(k, cache, cache.heads, "k")
    vp, vt, vh = _rows(v, cache, cache.heads, "v")
    rows = k.shape[0]
    if v.shape[0] != rows:
        raise ValueError(f"k and v must have the same rows, got {rows} and {v.shape[0]}")
    _one_each(k, s.n, cu, "k and v")
    if max_new is None:
        max_new = 1 if cu is None else rows
    with _on(cache.device):
        check(lib().int8_cache_write(_byref(cache._struct), _byref(s), kp, kt, kh, vp, vt, vh, rows,
                                     int(max_new), _stream(cache.device)))


def cache_read(cache, page_table, lengths, cu, total, slots=None, max_len=None, out=None):
    """Reads sequences back: (k, v) [total][heads][head_dim] of the cache's type;
    the tokens of sequence i are rows cu[i] .. cu[i] + lengths[i] - 1.  ``max_len``:
    at least the longest sequence (None: what the page table holds).  Rows that no
    sequence covers are not written."""
    s = _sequences(cache, page_table, lengths, cu, slots)
    shape = (int(total), cache.heads, cache.head_dim)
    if cu is None:
        raise ValueError("cu must name the first row of each sequence")
    k, v = (None, None) if out is None else out
    k, kp = _result(k, cache.dtype, shape, cache.device, "k")
    v, vp = _result(v, cache.dtype, shape, cache.device, "v")
    if max_len is None:
        max_len = s.max_pages * cache.page_size
    with _on(cache.device):
        check(lib().int8_cache_read(_byref(cache._struct), _byref(s), kp, vp, shape[0],
                                    int(max_len), _stream(cache.device)))
    return k, v


def attention_workspace_bytes(cache, n, q_heads, max_q, max_len, window=0):
    """Bytes of scratch that ``cache_attention`` uses for these sizes."""
    return int(lib().i8l_attention_workspace_bytes(_byref(cache._struct), n, q_heads, max_q,
                                                   max_len, window))


def cache_attention(q, cache, page_table, lengths, cu=None, slots=None, max_q=None, max_len=None,
                    scale=None, window=0, alibi=None, out=None, workspace=None):
    """Causal attention over a cache that already holds the queries' own tokens
    (``cache_write`` comes first): q [rows][q_heads][head_dim] -> the same shape.

    Row j of a sequence with m rows is the query of its token lengths - m + j and
    sees the tokens up to its own, with ``window`` > 0 only the last ``window`` of
    them; one with none to see gives 0.  q_heads is a multiple of the cache's heads
    (query head h reads kv head h // (q_heads / heads)).  ``scale`` defaults to
    head_dim ** -0.5; ``alibi`` fp32 [q_heads]: a linear position bias, -alibi[h]
    per token of distance.  ``max_q`` (None: 1 without cu, else all rows) is at
    least the rows of any one sequence, ``max_len`` (None: what the page table
    holds) the longest sequence; sequences, cu and slots as for ``cache_write``.
    ``workspace`` (uint8, ``attention_workspace_bytes``): None allocates it.
    """
    _inference(q, alibi)
    s = _sequences(cache, page_table, lengths, cu, slots)
    qp, qt, qh = _rows(q, cache, None, "q")
    rows, heads, D = q.shape
    dev = cache.device
    _one_each(q, s.n, cu, "q")
    if max_q is None:
        max_q = 1 if cu is None else max(rows, 1)
    if max_len is None:
        max_len = s.max_pages * cache.page_size
    out, op = _result(out, q.dtype, (rows, heads, D), dev, "out")
    need = 0 if workspace is not None else \
        attention_workspace_bytes(cache, s.n, heads, max_q, max_len, window)
    hold, ws, nb = _scratch(workspace, need, dev)
    with _on(dev):
        check(lib().int8_cache_attention(
            _byref(cache._struct), _byref(s), qp, qt, qh, heads, rows, int(max_q), int(max_len),
            float(D ** -0.5 if scale is None else scale), int(window),
            None if alibi is None else _dense(alibi, torch.float32, (heads,), dev, "alibi"),
            op, ws, nb, _stream(dev)))
    return out
