"""Rotary positions and drafted tokens over the 8-bit cache: the norm and rotation of
query and key heads (with its gradient), keys appended to the cache with both on the
way, and attention for trees of drafted tokens.  Marshalling only, as in serving.py:
every step runs in the HIP kernels of libint8lin.so (include/int8lin.h states the
formulas).

    rot = rotary(head_dim)                                          # frequencies
    q, k = rotate_heads(q, positions, rot, k=k, q_weight=wq, k_weight=wk)
    q = cache_append(cache, k, v, page_table, lengths, q=q, rotary=rot)  # into the cache
    # several drafted tokens a sequence, checked in one pass:
    positions, masks = tree_plan(parents, lengths, cu=cu)
    o = tree_attention(q, k, v, cache, page_table, lengths, masks, positions=positions, cu=cu)
    path, counts, lengths, token = tree_accept(parents, tokens, choices, lengths, cu=cu)
    cache_append(cache, k, v, page_table, lengths, cu=cu, counts=counts, index=path)

``module.RotateHeads`` is the norm and rotation with gradients through autograd; the
rest is for inference.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _binding
from ._binding import HeadsGradStruct, HeadsStruct, RotaryStruct, check, lib
from .serving import (_dense, _half_type, _inference, _one_each, _result, _scratch, _sequences,
                      _stream)

MAX_DRAFTS = 512   # of one sequence (I8L_MAX_DRAFTS)
_byref = ctypes.byref
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(device, f, *args):
    """f on the device's current stream, the device the current one for the call."""
    if device.index == _current():
        status = f(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            status = f(*args, _stream(device))
    if status:
        check(status)


class Rotary:
    """Rotary positions: pair i of a head at position p turns by p * freqs[i].

    ``freqs`` fp32 [pairs] on the GPU (``rotary`` makes the usual ones); the pairs are
    elements (i, i + pairs), or (2 i, 2 i + 1) if ``interleaved``; elements from 2 * pairs
    on stay as they are.  ``factor`` multiplies what turns.  It holds the tensor's address:
    its attributes do not change, and the tensor must not be given other storage.  A copy
    (copy.copy: over the same tensor; deepcopy, pickle: over one of its own) holds its own.
    """

    __slots__ = ("freqs", "interleaved", "factor", "device", "_struct")

    def __init__(self, freqs, interleaved=False, factor=1.0):
        n = freqs.numel() if isinstance(freqs, torch.Tensor) else 0
        at = _dense(freqs, torch.float32, (n,), None, "freqs")
        factor, interleaved = float(factor), bool(interleaved)
        if not math.isfinite(factor):
            raise ValueError(f"factor must be finite, got {factor}")
        _put_freqs(self, freqs)
        _put_interleaved(self, interleaved)
        _put_factor(self, factor)
        _put_device(self, freqs.device)
        _put_struct(self, RotaryStruct(at, n, interleaved, factor))

    def __setattr__(self, name, x):
        raise AttributeError(f"{name}: a Rotary does not change; make a new one")

    def __delattr__(self, name):
        raise AttributeError(f"{name}: a Rotary does not change")

    def __reduce__(self):
        return type(self), (self.freqs, self.interleaved, self.factor)


# what the constructor writes an unchanging object's attributes with
_put_freqs, _put_interleaved, _put_factor, _put_device, _put_struct = (
    Rotary.__dict__[name].__set__ for name in Rotary.__slots__)


def rotary(dim, base=10000.0, interleaved=False, scaling=None, scale=1.0, original=None, low=1.0,
           high=32.0, factor=None, device="cuda"):
    """A ``Rotary`` that turns the first ``dim`` elements (even) of a head, with
    frequencies base ** (-2 i / dim).

    ``scaling`` stretches them for contexts ``scale`` times as long as the ``original``:
      "linear"  all frequencies over scale (positions interpolated);
      "base"    base * scale ** (dim / (dim - 2)): the slowest pair over scale, the
                fastest as it was;
      "parts"   by the turns r_i that a pair makes over ``original`` tokens: those below
                ``low`` over scale, those above ``high`` as they were, between them a ramp
                that is linear in r_i (one in the pair's number, as some models have, is
                given to ``Rotary`` as frequencies); ``factor`` then defaults to
                1 + 0.1 ln(scale).
    """
    if dim < 0 or dim % 2:
        raise ValueError(f"dim must be even and at least 0, got {dim}")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f'scaling must be None, "linear", "base" or "parts", got {scaling!r}')
    if scaling is None and scale != 1.0:
        raise ValueError("scale without scaling")
    if not (base > 0 and scale > 0):
        raise ValueError("base and scale must be above 0")
    if scaling == "base" and dim > 2:
        base = base * scale ** (dim / (dim - 2))
    freqs = [base ** (-2.0 * i / dim) for i in range(dim // 2)] if dim else []
    if scaling == "linear":
        freqs = [f / scale for f in freqs]
    if scaling == "parts":
        if original is None or original <= 0 or not high > low:
            raise ValueError('"parts" needs the original length and high above low')
        keep = [min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for f in freqs]
        freqs = [f * (g + (1.0 - g) / scale) for f, g in zip(freqs, keep)]
        if factor is None and scale > 1.0:
            factor = 1.0 + 0.1 * math.log(scale)
    return Rotary(torch.tensor(freqs, dtype=torch.float32, device=device), interleaved,
                  1.0 if factor is None else factor)


def _turn(rot, device):
    """The struct's reference (None: nothing turns)."""
    if rot is None:
        return None
    if not isinstance(rot, Rotary):
        raise TypeError("rotary must be a Rotary")
    if rot.device != device:
        raise ValueError(f"rotary must be on {device} (got {rot.device})")
    return _byref(rot._struct)


def _heads(t, dtype, device, rows, heads, D, name):
    """(pointer, token stride, head stride) of a [rows][heads][D] tensor (None: any number);
    what is right is settled first, what is wrong said after, as in serving._dense."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.dim() == 3:
        n, h, d = t.shape
        if (rows is None or n == rows) and (heads is None or h == heads) and d == D:
            st, sh, sd = t.stride()
            if sd == 1 or D == 1:
                return t.data_ptr(), st, sh
            raise ValueError(f"{name} must be contiguous in its last dimension")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    shape = "][".join("any" if s is None else str(s) for s in (rows, heads, D))
    raise ValueError(f"{name} must be [{shape}], got {list(t.shape)}")


def _weight(w, dtype, D, device, name):
    return None if w is None else _dense(w, dtype, (D,), device, name)


def _side(x, weight, out, dtype, device, rows, D, name):
    """(struct, output) of one tensor of heads."""
    p, ts, hs = _heads(x, dtype, device, rows, None, D, name)
    H = x.shape[1]
    if out is None:
        out = torch.empty((rows, H, D), dtype=dtype, device=device)
        y, yts, yhs = out.data_ptr(), H * D, D
    else:
        y, yts, yhs = _heads(out, dtype, device, rows, H, D, name + "_out")
    return HeadsStruct(p, ts, hs, y, yts, yhs,
                                _weight(weight, dtype, D, device, name + "_weight"), H), out


def rotate_heads(q, positions, rotary=None, k=None, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
                 k_out=None):
    """Norm of each head and rotation to its row's position, queries and keys in one pass.

    q [rows][heads][head_dim] and k (None, or [rows][kv_heads][head_dim]) fp16 or bf16
    (strided views are fine: multiples of 8 elements), positions int32 [rows] -> q', or
    (q', k') with k.  With a weight ([head_dim], of their type) each head is first divided
    by its root mean square (over head_dim, plus eps under the root) and multiplied by it.
    ``rotary`` (a ``Rotary``; None: no rotation).  fp32 throughout, rounded once.
    ``q_out`` and ``k_out`` (which may be q and k) receive the results if given.
    """
    _inference(q, k, q_weight, k_weight)
    code = _half_type(q, "q", 3)
    rows, _, D = q.shape
    dev, dt = q.device, q.dtype
    qs, q_out = _side(q, q_weight, q_out, dt, dev, rows, D, "q")
    ks = None
    if k is not None:
        ks, k_out = _side(k, k_weight, k_out, dt, dev, rows, D, "k")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight or k_out without k")
    _call(dev, lib().int8_rotate_heads, _byref(qs), None if ks is None else _byref(ks), D, rows,
          _dense(positions, torch.int32, (rows,), dev, "positions"), _turn(rotary, dev), float(eps), code)
    return q_out if k is None else (q_out, k_out)


def _grad_side(dy, x, weight, out, dtype, device, rows, D, name):
    """(struct, dx, dweight) of one tensor of heads."""
    p, ts, hs = _heads(dy, dtype, device, rows, None, D, "d" + name)
    H = dy.shape[1]
    w = _weight(weight, dtype, D, device, name + "_weight")
    xp, xts, xhs, dw = None, 0, 0, None
    if weight is not None:
        if x is None:
            raise ValueError(f"{name} (the forward pass's input) is needed with {name}_weight")
        xp, xts, xhs = _heads(x, dtype, device, rows, H, D, name)
        dw = torch.empty((D,), dtype=dtype, device=device)
    if out is None:
        out = torch.empty((rows, H, D), dtype=dtype, device=device)
        y, yts, yhs = out.data_ptr(), H * D, D
    else:
        y, yts, yhs = _heads(out, dtype, device, rows, H, D, f"d{name}_out")
    return HeadsGradStruct(p, ts, hs, xp, xts, xhs, y, yts, yhs, w,
                                    None if dw is None else dw.data_ptr(), H), out, dw


def rotate_heads_backward(dq, positions, rotary=None, q=None, dk=None, k=None, q_weight=None,
                          k_weight=None, eps=1e-6, dq_out=None, dk_out=None, workspace=None):
    """The gradient of ``rotate_heads``: dq (and dk) of its outputs -> (dq, dk, dq_weight,
    dk_weight) of its inputs, None for what was not there.

    q and k, the forward pass's inputs, are needed where there is a weight.  Weight
    gradients are summed over rows and heads in a fixed order.  ``dq_out`` and ``dk_out``
    (which may be dq and dk) receive the results if given; ``workspace`` (uint8,
    ``rotate_heads_workspace_bytes``): None allocates it.  It has no gradient of its own.
    """
    _inference(dq, q, dk, k, q_weight, k_weight)
    code = _half_type(dq, "dq", 3)
    rows, H, D = dq.shape
    dev, dt = dq.device, dq.dtype
    qs, dq_out, dqw = _grad_side(dq, q, q_weight, dq_out, dt, dev, rows, D, "q")
    ks, dkw = None, None
    if dk is not None:
        ks, dk_out, dkw = _grad_side(dk, k, k_weight, dk_out, dt, dev, rows, D, "k")
    elif k_weight is not None or dk_out is not None:
        raise ValueError("k_weight or dk_out without dk")
    need = 0
    if workspace is None and (dqw is not None or dkw is not None):
        need = rotate_heads_workspace_bytes(rows, D)
    hold, ws, nb = _scratch(workspace, need, dev)
    _call(dev, lib().int8_rotate_heads_backward, _byref(qs), None if ks is None else _byref(ks), D, rows,
          _dense(positions, torch.int32, (rows,), dev, "positions"), _turn(rotary, dev), float(eps), code,
          ws, nb)
    return dq_out, dk_out, dqw, dkw


def rotate_heads_workspace_bytes(rows, head_dim):
    """Bytes of scratch that ``rotate_heads_backward`` uses where there is a weight."""
    return int(lib().i8l_rotate_heads_workspace_bytes(rows, head_dim))


def cache_append(cache, k, v, page_table, lengths, q=None, rotary=None, q_weight=None, k_weight=None,
                 eps=1e-6, cu=None, slots=None, max_new=None, counts=None, index=None, q_out=None):
    """``cache_write`` with the keys' norm and rotation on the way, and the queries' in the
    same launch: what ``rotate_heads`` at each row's own position and then ``cache_write``
    give, bit for bit.  Returns q' [rows][q_heads][head_dim] (None without q).

    Row j of a sequence with m rows is its token, and has the position, lengths - m + j.
    ``q_weight``, ``k_weight``, ``eps`` and ``rotary`` as for ``rotate_heads``; ``q_out``
    (which may be q) receives q' if given, rows outside the sequences are left as they
    are.  ``counts`` (int32 [n]): of sequence i only the first counts[i] rows from cu[i] on;
    ``index`` (int32 [rows]): row r of the call is row index[r] of k and v (without q) -
    the path of ``tree_accept``, say.  Everything else as for ``cache_write``.
    """
    _inference(q, k, v, q_weight, k_weight)
    s = _sequences(cache, page_table, lengths, cu, slots)
    D, dt, dev = cache.head_dim, cache.dtype, cache.device
    kp, kt, kh = _heads(k, dt, dev, None, cache.heads, D, "k")
    vp, vt, vh = _heads(v, dt, dev, k.shape[0], cache.heads, D, "v")
    kv_rows = k.shape[0]
    ip, rows = None, kv_rows
    if index is not None:
        if q is not None:
            raise ValueError("q and index: queries are not picked")
        if not isinstance(index, torch.Tensor):
            raise TypeError("index must be a torch.Tensor")
        rows = index.numel()
        ip = _dense(index, torch.int32, (rows,), dev, "index")
    if cu is None and rows != s.n:
        raise ValueError(f"k and v must have one row for each of the {s.n} sequences (or pass cu), "
                         f"got {rows}")
    qs = None
    if q is not None:
        qs, q_out = _side(q, q_weight, q_out, dt, dev, rows, D, "q")
    elif q_weight is not None or q_out is not None:
        raise ValueError("q_weight or q_out without q")
    if max_new is None:
        max_new = 1 if cu is None else rows
    _call(dev, lib().int8_cache_append, _byref(cache._struct), _byref(s),
          None if counts is None else _dense(counts, torch.int32, (s.n,), dev, "counts"), ip, kp, kt, kh,
          vp, vt, vh, kv_rows, rows, int(max_new), None if qs is None else _byref(qs),
          _weight(k_weight, dt, D, dev, "k_weight"), _turn(rotary, dev), float(eps))
    return q_out


def _tree(parents, lengths, cu, max_q):
    """(rows, n, max_q, device, pointers) of a tree's arrays."""
    if not isinstance(parents, torch.Tensor) or not isinstance(lengths, torch.Tensor):
        raise TypeError("parents and lengths must be torch.Tensors")
    rows, n, dev = parents.numel(), lengths.numel(), lengths.device
    lp = _dense(lengths, torch.int32, (n,), None, "lengths")
    pp = _dense(parents, torch.int32, (rows,), dev, "parents")
    cp = None if cu is None else _dense(cu, torch.int32, (n + 1,), dev, "cu")
    if cu is None and rows != n:
        raise ValueError(f"parents must have one row for each of the {n} sequences (or pass cu), "
                         f"got {rows}")
    if max_q is None:
        max_q = 1 if cu is None else min(max(rows, 1), MAX_DRAFTS)
    return rows, n, int(max_q), dev, (pp, lp, cp)


def tree_plan(parents, lengths, cu=None, max_q=None, positions=None, masks=None):
    """Positions and masks of drafted tokens, a tree of them behind each sequence.

    Row j of a sequence follows its row ``parents`` (int32 [rows]; counted within the
    sequence, an earlier one), or the cached text (-1, or no earlier row); lengths int32
    [n] counts the cached tokens, without drafts; cu int32 [n+1] as for ``cache_write``
    (None: one draft a sequence) -> (positions int32 [rows]: lengths + depth, masks int64
    [rows][words]: bit b of word w is draft 64 w + b of the sequence, set for the row
    itself and its ancestors).  ``max_q``: at least the drafts of any one sequence, at most
    512 (None: all rows, or 512; rows past it are not written).  ``positions`` and ``masks``
    receive the results if given.
    """
    rows, n, max_q, dev, (pp, lp, cp) = _tree(parents, lengths, cu, max_q)
    if masks is not None and (not isinstance(masks, torch.Tensor) or masks.dim() != 2):
        raise ValueError("masks must be an int64 tensor [rows][words]")
    words = -(-max_q // 64) if masks is None else masks.shape[1]
    positions, op = _result(positions, torch.int32, (rows,), dev, "positions")
    masks, mp = _result(masks, torch.int64, (rows, words), dev, "masks")
    _call(dev, lib().int8_tree_plan, pp, lp, cp, n, rows, max_q, op, mp, words)
    return positions, masks


def tree_workspace_bytes(cache, n, q_heads, max_q, max_len, window=0):
    """Bytes of scratch that ``tree_attention`` uses for these sizes."""
    return int(lib().i8l_tree_workspace_bytes(_byref(cache._struct), n, q_heads, max_q, max_len, window))


def tree_attention(q, k, v, cache, page_table, lengths, masks, positions=None, cu=None, slots=None,
                   max_q=None, max_len=None, scale=None, window=0, alibi=None, out=None,
                   workspace=None):
    """Attention of drafted tokens over a cache that does not hold them, and over the
    drafts that their masks name: q [rows][q_heads][head_dim] -> the same shape.

    k, v [rows][heads][head_dim]: the drafts' keys and values (turned already); lengths
    counts the cached tokens, which every draft of the sequence sees.  masks int64
    [rows][words] and positions int32 [rows] as ``tree_plan`` makes them (any masks will
    do); positions are needed with ``window`` (only keys less than that many positions
    before the draft's) or ``alibi``.  A row with nothing to see gives 0.  ``max_q`` (None: 1
    without cu, else all rows, or what masks have bits for): at least the drafts of any one
    sequence; drafts past it are neither seen nor answered.  Everything else, the workspace
    too (``tree_workspace_bytes``), as for ``cache_attention``.
    """
    _inference(q, k, v, alibi)
    s = _sequences(cache, page_table, lengths, cu, slots)
    D, dt, dev = cache.head_dim, cache.dtype, cache.device
    qp, qt, qh = _heads(q, dt, dev, None, None, D, "q")
    rows, heads, _ = q.shape
    kp, kt, kh = _heads(k, dt, dev, rows, cache.heads, D, "k")
    vp, vt, vh = _heads(v, dt, dev, rows, cache.heads, D, "v")
    _one_each(q, s.n, cu, "q")
    if not isinstance(masks, torch.Tensor) or masks.dim() != 2:
        raise ValueError("masks must be an int64 tensor [rows][words]")
    words = masks.shape[1]
    if max_q is None:
        max_q = 1 if cu is None else max(min(rows, 64 * words), 1)
    if max_len is None:
        max_len = s.max_pages * cache.page_size
    out, op = _result(out, dt, (rows, heads, D), dev, "out")
    need = 0 if workspace is not None else \
        tree_workspace_bytes(cache, s.n, heads, max_q, max_len, window)
    hold, ws, nb = _scratch(workspace, need, dev)
    _call(dev, lib().int8_tree_attention, _byref(cache._struct), _byref(s), qp, qt, qh, heads, kp, kt, kh,
          vp, vt, vh, rows, int(max_q), int(max_len),
          _dense(masks, torch.int64, (rows, words), dev, "masks"), words,
          None if positions is None else _dense(positions, torch.int32, (rows,), dev, "positions"),
          float(D ** -0.5 if scale is None else scale), int(window),
          None if alibi is None else _dense(alibi, torch.float32, (heads,), dev, "alibi"), op, ws, nb)
    return out


def tree_accept(parents, tokens, choices, lengths, cu=None, first=None, max_q=None):
    """The drafts that the model's choices accept: (path int32 [rows], counts int32 [n],
    lengths int32 [n], next int64 [n]).

    tokens int64 [rows]: the drafted tokens; choices int64 [rows]: the token that the model
    chooses to follow each of them.  ``first`` int64 [n]: the token that follows each
    sequence's cached text; None: row 0 of each sequence is that token and accepted.  From
    an accepted draft the path goes on to its first child that is the chosen token.
    path[cu[i]] .. hold the rows of sequence i's accepted drafts, then -1; counts their
    number; lengths the old ones plus counts; next the token chosen after the last.
    path, counts and the new lengths are what ``cache_append`` takes as index, counts
    and lengths.  parents, lengths, cu and max_q as for ``tree_plan``.
    """
    rows, n, max_q, dev, (pp, lp, cp) = _tree(parents, lengths, cu, max_q)
    # (one allocation: path, counts, lengths)
    ints = torch.empty((rows + 2 * n,), dtype=torch.int32, device=dev)
    path, counts, longer = ints.split([rows, n, n])
    after = torch.empty((n,), dtype=torch.int64, device=dev)
    at = ints.data_ptr()
    _call(dev, lib().int8_tree_accept, pp, _dense(tokens, torch.int64, (rows,), dev, "tokens"),
          _dense(choices, torch.int64, (rows,), dev, "choices"),
          None if first is None else _dense(first, torch.int64, (n,), dev, "first"), lp, cp, n, rows, max_q,
          at, at + 4 * rows, at + 4 * (rows + n), after.data_ptr())
    return path, counts, longer, after
