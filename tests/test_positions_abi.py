"""Rotary positions and drafts, checks that need no GPU: arguments are refused on the
host before any HIP call, the frequencies, and the oracle's functions against brute
force and differences."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from oracle import positions_oracle as O  # noqa: E402
from test_serving_abi import BAD_CACHES, BAD_SEQS, cache_struct, seqs_struct  # noqa: E402

OK, INVALID, WORKSPACE = 0, 1, 3
P16 = 0x10000   # fake, 16-byte aligned, never dereferenced
P8 = P16 + 8
ref = ctypes.byref


def rotary_struct(**kw):
    from mixed_precision_quantized_int8_amd import _binding

    a = dict(freqs=P16, pairs=32, interleaved=0, factor=1.0)
    a.update(kw)
    return _binding.RotaryStruct(*[a[n] for n, _ in _binding.RotaryStruct._fields_])


def heads_struct(**kw):
    from mixed_precision_quantized_int8_amd import _binding

    a = dict(x=P16, x_token_stride=256, x_head_stride=64, y=P16, y_token_stride=256, y_head_stride=64,
             weight=P16, heads=4)
    a.update(kw)
    return _binding.HeadsStruct(*[a[n] for n, _ in _binding.HeadsStruct._fields_])


def grad_struct(**kw):
    from mixed_precision_quantized_int8_amd import _binding

    a = dict(dy=P16, dy_token_stride=256, dy_head_stride=64, x=P16, x_token_stride=256, x_head_stride=64,
             dx=P16, dx_token_stride=256, dx_head_stride=64, weight=P16, dweight=P16, heads=4)
    a.update(kw)
    return _binding.HeadsGradStruct(*[a[n] for n, _ in _binding.HeadsGradStruct._fields_])


BAD_ROTARY = [dict(freqs=None), dict(freqs=P16 + 2), dict(pairs=-1), dict(pairs=33), dict(interleaved=2),
              dict(interleaved=-1), dict(factor=math.nan), dict(factor=math.inf)]
BAD_HEADS = [dict(y_head_stride=56), dict(y_token_stride=0), dict(y_token_stride=248), dict(x=None), dict(x=P8), dict(y=None), dict(y=P8), dict(x_token_stride=4),
             dict(x_head_stride=-8), dict(y_token_stride=-8), dict(y_head_stride=12), dict(weight=P8),
             dict(heads=0), dict(heads=65537)]


def test_rotate_heads_refusals(i8l):
    L = i8l.lib()

    def call(q=None, k=None, D=64, rows=2, pos=P16, rot=None, eps=1e-6, dtype=0, none=()):
        return L.int8_rotate_heads(None if "q" in none else ref(q or heads_struct()),
                                   None if k is None else ref(k), D, rows, pos,
                                   ref(rot or rotary_struct()), eps, dtype, None)

    for bad in (dict(none=("q",)), dict(D=0), dict(D=24), dict(D=272), dict(rows=-1), dict(rows=1 << 31),
                dict(pos=None), dict(pos=P16 + 2), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
                dict(dtype=2), dict(dtype=-1), dict(rows=1 << 30)):
        assert call(**bad) == INVALID, bad
        assert "int8_rotate_heads: " in i8l.last_error()
    for bad in BAD_ROTARY:
        assert call(rot=rotary_struct(**bad)) == INVALID, bad
    for bad in BAD_HEADS:
        assert call(q=heads_struct(**bad)) == INVALID, bad
        assert call(k=heads_struct(**bad)) == INVALID, bad
    assert call(rows=0, q=heads_struct(x=None)) == OK and i8l.last_error() == ""
    # heads outside tokens do not overlap either (refused for the positions here)
    assert call(q=heads_struct(y_token_stride=64, y_head_stride=128), pos=None) == INVALID
    assert "positions" in i8l.last_error()
    assert call(rows=0, rot=rotary_struct(pairs=0, freqs=None)) == OK


def test_rotate_heads_backward_refusals(i8l):
    L = i8l.lib()
    need = L.i8l_rotate_heads_workspace_bytes(100, 64)
    assert need > 0

    def call(q=None, k=None, D=64, rows=100, pos=P16, rot=None, eps=1e-6, dtype=0, ws=P16, n=need):
        return L.int8_rotate_heads_backward(ref(q or grad_struct()), None if k is None else ref(k), D, rows,
                                            pos, ref(rot or rotary_struct()), eps, dtype, ws, n, None)

    for bad in (dict(D=24), dict(rows=-1), dict(pos=None), dict(eps=-1.0), dict(dtype=3), dict(ws=None),
                dict(ws=P8), dict(rows=1 << 30)):
        assert call(**bad) == INVALID, bad
    assert call(n=need - 1) == WORKSPACE and str(need) in i8l.last_error()
    for bad in BAD_ROTARY:
        assert call(rot=rotary_struct(**bad)) == INVALID, bad
    for bad in (dict(dy=None), dict(dy=P8), dict(dx=None), dict(x=None), dict(x=P8), dict(weight=P8),
                dict(dweight=None), dict(dweight=P16 + 1), dict(heads=0), dict(dy_token_stride=3),
                dict(x_head_stride=-8), dict(dx_token_stride=4), dict(dx_head_stride=0),
                dict(dx_token_stride=128)):
        assert call(q=grad_struct(**bad)) == INVALID, bad
        assert call(k=grad_struct(**bad)) == INVALID, bad
    assert L.int8_rotate_heads_backward(None, None, 64, 2, P16, ref(rotary_struct()), 1e-6, 0, None, 0,
                                        None) == INVALID
    # without weights: no input, no workspace; without rows nothing to do
    assert call(q=grad_struct(weight=None, dweight=None, x=None), rows=0, ws=None, n=0) == OK
    assert L.i8l_rotate_heads_workspace_bytes(100, 24) == 0
    assert L.i8l_rotate_heads_workspace_bytes(-1, 64) == 0


def test_cache_append_refusals(i8l):
    L = i8l.lib()

    def call(cache=None, seqs=None, counts=None, index=None, k=P16, kt=256, kh=64, v=P16, vt=256, vh=64,
             kv_rows=2, rows=2, most=1, q=None, kw=P16, rot=None, eps=1e-6):
        return L.int8_cache_append(ref(cache or cache_struct()), ref(seqs or seqs_struct()), counts, index, k,
                                   kt, kh, v, vt, vh, kv_rows, rows, most,
                                   None if q is None else ref(q), kw, ref(rot or rotary_struct()), eps, None)

    for bad in BAD_CACHES:
        assert call(cache=cache_struct(**bad)) == INVALID, bad
    for bad in BAD_SEQS:
        assert call(seqs=seqs_struct(**bad)) == INVALID, bad
    for bad in BAD_ROTARY:
        assert call(rot=rotary_struct(**bad)) == INVALID, bad
    for bad in BAD_HEADS:
        assert call(q=heads_struct(**bad)) == INVALID, bad
    for bad in (dict(counts=P16 + 2), dict(index=P16 + 2), dict(index=P16, q=heads_struct()), dict(k=None),
                dict(k=P8), dict(v=P8), dict(kt=4), dict(kh=12), dict(vt=-8), dict(kv_rows=1),
                dict(kv_rows=0, index=P16), dict(rows=-1), dict(rows=1 << 40), dict(kv_rows=-1),
                dict(most=-1), dict(kw=P8), dict(eps=-1.0), dict(seqs=seqs_struct(max_pages=0))):
        assert call(**bad) == INVALID, bad
        assert "int8_cache_append: " in i8l.last_error()
    assert call(rows=0) == OK and call(most=0) == OK and call(seqs=seqs_struct(n=0)) == OK
    c, s = cache_struct(heads=4096), seqs_struct(max_pages=1 << 20)
    most = 2046 * 16 + 16
    assert call(cache=c, seqs=s, rows=most, kv_rows=most, most=most) == INVALID
    assert "too many" in i8l.last_error()
    assert call(seqs=s, rows=1 << 27, kv_rows=1 << 27, most=1 << 27, q=heads_struct(heads=64, y_token_stride=4096)) == INVALID
    assert "too many" in i8l.last_error()


def test_tree_refusals(i8l):
    L = i8l.lib()

    def plan(parents=P16, lengths=P16, cu=P16, n=2, rows=5, max_q=4, pos=P16, masks=P16, words=1):
        return L.int8_tree_plan(parents, lengths, cu, n, rows, max_q, pos, masks, words, None)

    for bad in (dict(parents=None), dict(parents=P16 + 1), dict(lengths=None), dict(cu=P16 + 2), dict(n=-1),
                dict(n=65536), dict(rows=-1), dict(rows=1 << 31), dict(max_q=0), dict(max_q=513, words=8),
                dict(max_q=65), dict(words=0), dict(words=9), dict(pos=None), dict(masks=None),
                dict(masks=P16 + 4)):
        assert plan(**bad) == INVALID, bad
    assert plan(n=0) == OK and plan(rows=0) == OK and i8l.last_error() == ""

    def accept(parents=P16, tokens=P16, choices=P16, first=None, lengths=P16, cu=P16, n=2, rows=5, max_q=4,
               path=P16, counts=P16, longer=P16, after=P16):
        return L.int8_tree_accept(parents, tokens, choices, first, lengths, cu, n, rows, max_q, path, counts,
                                  longer, after, None)

    for bad in (dict(parents=None), dict(tokens=None), dict(tokens=P16 + 4), dict(choices=None),
                dict(first=P16 + 4), dict(lengths=None), dict(cu=P16 + 2), dict(n=-1), dict(rows=-1),
                dict(max_q=0), dict(max_q=513), dict(path=None), dict(counts=None), dict(longer=P16 + 2),
                dict(after=P16 + 4)):
        assert accept(**bad) == INVALID, bad
    assert accept(n=0) == OK

    def attend(cache=None, seqs=None, q=P16, qt=512, qh=64, heads=8, k=P16, kt=256, kh=64, v=P16, vt=256,
               vh=64, rows=2, max_q=1, max_len=80, masks=P16, words=1, pos=P16, scale=0.125, window=0,
               alibi=None, out=P16, ws=None, n=0):
        return L.int8_tree_attention(ref(cache or cache_struct()), ref(seqs or seqs_struct()), q, qt, qh, heads,
                                     k, kt, kh, v, vt, vh, rows, max_q, max_len, masks, words, pos, scale,
                                     window, alibi, out, ws, n, None)

    for bad in BAD_CACHES:
        assert attend(cache=cache_struct(**bad)) == INVALID, bad
    for bad in BAD_SEQS:
        assert attend(seqs=seqs_struct(**bad)) == INVALID, bad
    for bad in (dict(q=None), dict(q=P8), dict(qt=9), dict(qh=-8), dict(heads=0), dict(heads=6), dict(k=None),
                dict(kt=4), dict(v=P8), dict(vh=-8), dict(rows=-1), dict(rows=1 << 40), dict(max_q=0),
                dict(max_q=65), dict(max_q=513, words=8), dict(max_len=-1), dict(masks=None),
                dict(masks=P16 + 4), dict(words=0), dict(words=9), dict(pos=None, window=5),
                dict(pos=None, alibi=P16), dict(pos=P16 + 2), dict(scale=math.nan), dict(window=-1),
                dict(alibi=P16 + 1), dict(out=None), dict(out=P8), dict(seqs=seqs_struct(max_pages=0))):
        assert attend(**bad) == INVALID, bad
        assert "int8_tree_attention: " in i8l.last_error()
    need = L.i8l_tree_workspace_bytes(ref(cache_struct()), 2, 8, 1, 100000, 0)
    assert need > 0 and L.i8l_tree_workspace_bytes(ref(cache_struct()), 2, 8, 1, 100, 0) == 0
    assert L.i8l_tree_workspace_bytes(ref(cache_struct()), 2, 8, 513, 100000, 0) == 0
    assert attend(max_len=100000) == INVALID and "workspace is NULL" in i8l.last_error()
    assert attend(max_len=100000, ws=P16, n=need - 1) == WORKSPACE
    assert attend(rows=0) == OK and attend(seqs=seqs_struct(n=0)) == OK


def test_wrappers_refuse(i8l):
    x = torch.zeros((2, 4, 64), dtype=torch.float16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        i8l.rotate_heads(x, pos)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        i8l.rotate_heads(x.float(), pos)
    with pytest.raises(RuntimeError, match="gradient"):
        i8l.rotate_heads(x.clone().requires_grad_(), pos)
    with pytest.raises(ValueError, match="on a GPU"):
        i8l.rotate_heads_backward(x, pos)
    with pytest.raises(ValueError, match="on a GPU"):
        i8l.Rotary(torch.ones(4))
    with pytest.raises(TypeError, match="float32"):
        i8l.Rotary(torch.ones(4, dtype=torch.float64))
    with pytest.raises(TypeError, match="KVCache"):
        i8l.cache_append(x, x, x, torch.zeros((1, 1), dtype=torch.int32), pos)
    with pytest.raises(TypeError, match="KVCache"):
        i8l.tree_attention(x, x, x, x, torch.zeros((1, 1), dtype=torch.int32), pos, pos)
    with pytest.raises(TypeError):
        i8l.tree_plan([0], pos)
    with pytest.raises(ValueError, match="on a GPU"):
        i8l.tree_plan(pos, pos)
    with pytest.raises(ValueError, match="on a GPU"):
        i8l.tree_accept(pos, pos, pos, pos)


def test_rotary_refuses_and_scales(i8l, monkeypatch):
    """The frequencies of each way of stretching them, by hand."""
    from mixed_precision_quantized_int8_amd import positions

    made = []
    monkeypatch.setattr(positions, "Rotary", lambda f, i, factor: made.append((f, i, factor)))

    def freqs(*a, **kw):
        positions.rotary(*a, device="cpu", **kw)
        return made[-1]

    for bad in (dict(dim=3), dict(dim=-2), dict(dim=8, scaling="other"), dict(dim=8, scale=2.0),
                dict(dim=8, scaling="parts", scale=2.0), dict(dim=8, base=0.0),
                dict(dim=8, scaling="linear", scale=0.0),
                dict(dim=8, scaling="parts", scale=2.0, original=100, low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            freqs(**bad)
    f, inter, factor = freqs(8, interleaved=True)
    assert inter and factor == 1.0 and f.dtype == torch.float32
    want = [1.0, 0.1, 0.01, 0.001]
    assert torch.equal(f, torch.tensor(want))
    assert torch.equal(freqs(8, scaling="linear", scale=4.0)[0], torch.tensor([w / 4 for w in want]))
    f = freqs(8, scaling="base", scale=4.0)[0].double()
    # (a rounding to fp32, 2^-24)
    assert f[0] == 1.0 and abs(f[-1] - 0.001 / 4) < 2 ** -23 * 0.00025   # the slowest pair exactly over scale
    assert bool((f[1:-1] > torch.tensor(want[1:-1]) / 4).all()) and bool((f[1:-1] < torch.tensor(want[1:-1])).all())
    # 628 tokens: the pairs turn 100, 10, 1 and 0.1 times (over 2 pi: 628 f / 6.28)
    f, _, factor = freqs(8, scaling="parts", scale=4.0, original=200 * math.pi, low=1.0, high=19.0)
    assert abs(factor - (1 + 0.1 * math.log(4))) < 1e-12
    got = f.double() / torch.tensor(want, dtype=torch.float64)
    assert float((got - torch.tensor([1.0, 0.5 + 0.5 / 4, 0.25, 0.25], dtype=torch.float64)).abs().max()) < 1e-6
    assert freqs(8, scaling="parts", scale=4.0, original=100, factor=2.0)[2] == 2.0
    assert freqs(0)[0].numel() == 0


# ---- the oracle -------------------------------------------------------------------


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_turn_by_hand(interleaved):
    x = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0, 6.0], dtype=torch.float64).view(1, 1, 6)
    f = torch.tensor([math.pi / 2, math.pi])
    y = O.turn(x, torch.tensor([1]), f, interleaved, 2.0)[0, 0]
    a = [2 * v for v in ([-2, 1, -3, -4] if interleaved else [-3, -2, 1, -4])] + [5, 6]
    assert float((y - torch.tensor(a, dtype=torch.float64)).abs().max()) < 1e-5   # (pi in fp32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs", [0, 3, 8])
def test_oracle_gradient_by_differences(interleaved, pairs):
    g = torch.Generator().manual_seed(pairs)
    x = torch.randn((3, 2, 16), generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(16, generator=g, dtype=torch.float64)
    f = torch.rand(pairs, generator=g)
    pos = torch.tensor([0, 5, -77])
    dy = torch.randn(x.shape, generator=g, dtype=torch.float64)

    def loss(x, w):
        return float((O.turn(O.norm(x, w, 1e-3), pos, f, interleaved, 1.3) * dy).sum())

    (dx, _), (dw, _) = O.rotate_grad(dy, x, pos, f, interleaved, 1.3, w, 1e-3)
    h = 1e-5
    for t, d in ((x, dx), (w, dw)):
        flat = t.view(-1)
        for i in range(0, flat.numel(), 5):
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss(x, w)
            flat[i] = keep - h
            down = loss(x, w)
            flat[i] = keep
            # central differences: h^2 times third derivatives (below 100 here), 2^-52 / h of the loss
            assert abs((up - down) / (2 * h) - float(d.reshape(-1)[i])) < 1e-7


def test_oracle_zero_head_is_zero():
    y, tol = O.rotate(torch.zeros((2, 1, 16), dtype=torch.float16), torch.tensor([1, 2]),
                      torch.ones(4), weight=torch.ones(16).half(), eps=0.0)
    assert bool((y == 0).all())


def test_oracle_tree_by_hand():
    # 0 - 1 - 3, 0 - 2, 4 behind the text again, 5 with a parent that is not before it
    parents = [-1, 0, 0, 1, -1, 9]
    positions, seen = O.tree_plan(parents, 10)
    assert positions == [10, 11, 11, 12, 10, 10]
    assert seen == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {4}, {5}]
    assert O.words(seen, 1)[:, 0].tolist() == [1, 3, 5, 11, 16, 32]
    assert O.words([{63, 64}], 2).tolist() == [[-(1 << 63), 1]]
    tokens, choices = [7, 8, 9, 5, 6, 6], [9, 1, 2, 3, 4, 4]
    assert O.tree_accept(parents, tokens, choices) == ([0, 2], 2)
    assert O.tree_accept(parents, tokens, choices, first=6) == ([4], 4)
    assert O.tree_accept(parents, tokens, choices, first=1) == ([], 1)
    assert O.tree_accept([], [], []) == ([], -1)


def test_oracle_tree_attention_is_causal_attention_on_a_chain():
    """A chain of drafts sees what a run of queries sees."""
    from oracle import serving_oracle as S

    g = torch.Generator().manual_seed(1)
    m, n, H, G, D = 4, 9, 2, 2, 16
    q = torch.randn((m, H * G, D), generator=g)
    k, v = torch.randn((n, H, D), generator=g), torch.randn((n, H, D), generator=g)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625])
    back = torch.arange(n - m, n)[:, None] - torch.arange(n)[None]
    a, _ = S.attention(q, k, v, 0.3, 3, slopes)
    b, tol = O.tree_attention(q, k, v, 0.3, (back >= 0) & (back < 3), back, slopes)
    assert float((a - b).abs().max()) < 1e-12 and bool((tol > 0).all())
    o, t = O.tree_attention(q, k, v, 0.3, torch.zeros((m, n), dtype=torch.bool))
    assert bool((o == 0).all()) and bool((t == 0).all())
