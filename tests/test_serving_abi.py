"""Serving operators, checks that need no GPU: arguments are refused on the host
before any HIP call, and the oracle's functions against brute force."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import int8_oracle  # noqa: E402
from oracle import serving_oracle as O  # noqa: E402

OK, INVALID, K_TOO_LARGE, WORKSPACE = 0, 1, 2, 3
P16 = 0x10000   # fake, 16-byte aligned, never dereferenced
P8 = P16 + 8


def cache_struct(**kw):
    from mixed_precision_quantized_int8_amd import _binding

    a = dict(k_codes=P16, v_codes=P16, k_scale=P16, v_scale=P16, k_tail=P16, v_tail=P16,
             n_pages=10, n_slots=2, heads=4, head_dim=64, page_size=16, dtype=0)
    a.update(kw)
    return _binding.KVCacheStruct(*[a[n] for n, _ in _binding.KVCacheStruct._fields_])


def seqs_struct(**kw):
    from mixed_precision_quantized_int8_amd import _binding

    a = dict(page_table=P16, lengths=P16, cu=P16, slots=P16, n=2, max_pages=5)
    a.update(kw)
    return _binding.SequencesStruct(*[a[n] for n, _ in _binding.SequencesStruct._fields_])


def test_rmsnorm_quant_refusals(i8l):
    L = i8l.lib()

    def call(X=P16, R=P16, W=P16, M=4, K=64, eps=1e-5, dtype=0, Xq=P16, sx=P16, h=P16):
        return L.int8_rmsnorm_quant(X, R, W, M, K, eps, dtype, Xq, sx, h, None)

    for bad in (dict(X=None), dict(X=P8), dict(R=P8), dict(W=P8), dict(h=P8), dict(Xq=None),
                dict(Xq=P8), dict(sx=None), dict(sx=P16 + 2), dict(K=72), dict(K=0), dict(K=8),
                dict(M=-1), dict(dtype=2), dict(dtype=-1), dict(eps=-1.0), dict(eps=math.nan),
                dict(eps=math.inf)):
        assert call(**bad) == INVALID, bad
        assert "int8_rmsnorm_quant: " in i8l.last_error()
    assert call(K=133152) == K_TOO_LARGE
    assert call(M=0, X=None) == OK and i8l.last_error() == ""


def test_linear_codes_refusals(i8l):
    L = i8l.lib()

    def call(Xq=P16, sx=P16, M=4, K=64, Wq=P16, sw=P16, N=32, b=P16, Y=P16, ws=None, n=0):
        return L.int8_linear_codes(Xq, sx, M, K, Wq, sw, N, b, Y, ws, n, None)

    for bad in (dict(Xq=None), dict(Xq=P8), dict(sx=None), dict(Wq=None), dict(Wq=P8),
                dict(sw=P16 + 1), dict(Y=None), dict(Y=P8), dict(b=P16 + 1), dict(K=24),
                dict(M=-1), dict(N=-1), dict(ws=P8, n=1 << 30)):
        assert call(**bad) == INVALID, bad
    assert call(K=133152) == K_TOO_LARGE
    need = i8l.lib().i8l_codes_workspace_bytes(520, 2048, 1300)
    assert need == 2 * 520 * 1300 * 4           # 105 tiles of 128 x 64, split in two
    # 1344 tiles of 256 x 256: the last 64 split in four
    assert i8l.lib().i8l_codes_workspace_bytes(2048, 14336, 43008) == 64 * 4 * 256 * 256 * 4
    assert call(M=520, K=2048, N=1300, ws=P16, n=need - 1) == WORKSPACE
    assert str(need) in i8l.last_error()
    assert L.i8l_codes_workspace_bytes(256, 4096, 16384) == 0
    assert L.i8l_codes_workspace_bytes(4, 70, 4) == 0
    assert call(M=0) == OK and call(N=0) == OK


BAD_CACHES = [dict(k_codes=None), dict(v_codes=P8), dict(k_scale=None), dict(v_scale=P16 + 2),
              dict(k_tail=None), dict(v_tail=P8), dict(n_pages=0), dict(n_slots=0),
              dict(n_pages=1 << 31), dict(heads=0), dict(heads=4097), dict(head_dim=24),
              dict(head_dim=0), dict(head_dim=272), dict(page_size=8), dict(page_size=48),
              dict(page_size=256), dict(dtype=3)]
BAD_SEQS = [dict(page_table=None), dict(lengths=None), dict(lengths=P16 + 1), dict(n=-1),
            dict(n=65536), dict(max_pages=-1), dict(max_pages=1 << 26), dict(slots=P16 + 2),
            dict(cu=P16 + 2)]


def test_cache_calls_refuse(i8l):
    L, ref = i8l.lib(), ctypes.byref

    def write(cache=None, seqs=None, k=P16, kt=256, kh=64, v=P16, vt=256, vh=64, rows=2, most=1):
        return L.int8_cache_write(ref(cache or cache_struct()), ref(seqs or seqs_struct()), k, kt,
                                  kh, v, vt, vh, rows, most, None)

    def read(cache=None, seqs=None, k=P16, v=P16, rows=2, most=1):
        return L.int8_cache_read(ref(cache or cache_struct()), ref(seqs or seqs_struct()), k, v,
                                 rows, most, None)

    def attend(cache=None, seqs=None, q=P16, qt=512, qh=64, heads=8, rows=2, max_q=1, max_len=80,
               scale=0.125, window=0, alibi=None, out=P16, ws=None, n=0):
        return L.int8_cache_attention(ref(cache or cache_struct()), ref(seqs or seqs_struct()), q,
                                      qt, qh, heads, rows, max_q, max_len, scale, window, alibi,
                                      out, ws, n, None)

    for f in (write, read, attend):
        for bad in BAD_CACHES:
            assert f(cache=cache_struct(**bad)) == INVALID, (f, bad)
        for bad in BAD_SEQS:
            assert f(seqs=seqs_struct(**bad)) == INVALID, (f, bad)
        assert f(rows=-1) == INVALID and f(rows=1 << 40) == INVALID
        assert f(rows=0) == OK and f(seqs=seqs_struct(n=0)) == OK
    assert L.int8_cache_write(None, ref(seqs_struct()), P16, 256, 64, P16, 256, 64, 2, 1,
                              None) == INVALID
    assert L.int8_cache_read(ref(cache_struct()), None, P16, P16, 2, 1, None) == INVALID
    assert read(seqs=seqs_struct(cu=None)) == INVALID and "cu is NULL" in i8l.last_error()
    for bad in (dict(k=None), dict(k=P8), dict(v=P8), dict(kt=4), dict(kh=12), dict(vt=-8),
                dict(most=-1)):
        assert write(**bad) == INVALID, bad
    for bad in (dict(k=None), dict(v=P8), dict(most=-1)):
        assert read(**bad) == INVALID, bad
    for bad in (dict(q=None), dict(q=P8), dict(qt=9), dict(qh=-8), dict(heads=0), dict(heads=6),
                dict(max_q=0), dict(max_len=-1), dict(window=-1), dict(scale=math.nan),
                dict(scale=math.inf), dict(out=None), dict(out=P8), dict(alibi=P16 + 1),
                dict(max_q=1 << 29, heads=8), dict(seqs=seqs_struct(max_pages=0))):
        assert attend(**bad) == INVALID, bad
    # a long context is split over workgroups: their partial results need a workspace
    need = L.i8l_attention_workspace_bytes(ref(cache_struct()), 2, 8, 1, 100000, 0)
    assert need > 0
    assert attend(max_len=100000) == INVALID and "workspace is NULL" in i8l.last_error()
    assert attend(max_len=100000, ws=P8, n=need) == INVALID
    assert attend(max_len=100000, ws=P16, n=need - 1) == WORKSPACE
    assert L.i8l_attention_workspace_bytes(ref(cache_struct()), 2, 8, 1, 100, 0) == 0
    assert L.i8l_attention_workspace_bytes(ref(cache_struct(head_dim=24)), 2, 8, 1, 100000, 0) == 0


def test_cache_calls_refuse_launches_that_are_too_large(i8l):
    """2^24 workgroups (pages x heads x 2) and more of one sequence in one call."""
    L, ref = i8l.lib(), ctypes.byref
    c, s = cache_struct(heads=4096), seqs_struct(max_pages=1 << 20)
    most = 2046 * 16 + 16   # pages + 2 reach 2^24 / (2 * 4096) = 2048 with the last token
    assert L.int8_cache_write(ref(c), ref(s), P16, 1 << 18, 64, P16, 1 << 18, 64, most, most,
                              None) == INVALID
    assert "too many" in i8l.last_error()
    assert L.int8_cache_read(ref(c), ref(s), P16, P16, most, 1 << 23, None) == INVALID
    assert "too many" in i8l.last_error()


def test_wrappers_refuse(i8l):
    X = torch.zeros((2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="on a GPU"):
        i8l.rmsnorm_quant(X)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        i8l.rmsnorm_quant(X.float())
    with pytest.raises(TypeError):
        i8l.linear_codes(X, None, None, None)
    c = torch.zeros((3, 2, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError, match="on a GPU"):
        i8l.new_cache(3, 1, 2, 64, 16, device="cpu")
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        i8l.KVCache(c, c, c, c, c, c)
    with pytest.raises(TypeError, match="KVCache"):
        i8l.cache_write(c, c, c, torch.zeros((1, 1), dtype=torch.int32), None)


# ---- the oracle -------------------------------------------------------------------


def test_oracle_codes_match_the_layers():
    """The same codes as the layer's row codes (no outlier columns)."""
    g = torch.Generator().manual_seed(0)
    X = torch.randn((7, 96), generator=g).half()
    X[2] = 0
    q, _, h = O.rmsnorm_quant(X)
    ref = int8_oracle.int8_linear(X.numpy(), np.zeros((16, 96), np.int8), np.zeros(16, np.float32),
                                  np.zeros((96, 16), np.float16), 0.0)
    assert np.array_equal(q.numpy(), ref["Xq"])


def test_oracle_norm_by_hand():
    X = torch.tensor([[3.0, -4.0] + [0.0] * 14], dtype=torch.float16)
    W = torch.full((16,), 2.0, dtype=torch.float16)
    q, s, h = O.rmsnorm_quant(X, W, residual=X, eps=0.0)
    assert h[0, :2].tolist() == [6.0, -8.0]
    assert q[0, :3].tolist() == [95, -127, 0]           # 12 * 127 / 16 = 95.25
    assert abs(float(s[0]) - 16.0 / math.sqrt(100.0 / 16)) < 1e-12


def test_oracle_page_by_hand():
    c, s = O.Store(2).page(torch.tensor([[1.0, -2.0], [0.5, 4.0]], dtype=torch.float16))
    assert c.tolist() == [[32, -64], [16, 127]]         # 31.75, -63.5 (away from 0), 15.875
    assert float(s) == float(np.float32(4.0) / np.float32(127.0))
    assert math.isnan(float(O.Store(2).page(torch.tensor([[1.0, math.inf]]).half())[1]))
    val, pages = O.Store(2).sequence(torch.ones((3, 1, 2), dtype=torch.float16) * 3)
    assert len(pages) == 1 and float(val[2, 0, 0]) == 3.0


@pytest.mark.parametrize("window", [0, 2])
def test_oracle_attention_by_brute_force(window):
    g = torch.Generator().manual_seed(1)
    m, n, H, G, D = 3, 5, 2, 2, 16
    q = torch.randn((m, H * G, D), generator=g)
    k, v = torch.randn((n, H, D), generator=g), torch.randn((n, H, D), generator=g)
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625])
    out, tol = O.attention(q, k, v, 0.3, window, slopes)
    for i in range(m):
        pos = n - m + i
        for h in range(H * G):
            num, den = [0.0] * D, 0.0
            for t in range(n):
                if t > pos or (window and pos - t >= window):
                    continue
                s = 0.3 * sum(float(q[i, h, d]) * float(k[t, h // G, d]) for d in range(D))
                w = math.exp(s - float(slopes[h]) * (pos - t))
                den += w
                for d in range(D):
                    num[d] += w * float(v[t, h // G, d])
            for d in range(D):
                assert abs(num[d] / den - float(out[i, h, d])) < 1e-12
    assert bool((tol > 0).all()) and float(tol.max()) < 0.02


def test_oracle_attention_with_nothing_to_see():
    out, _ = O.attention(torch.ones((3, 1, 16)), torch.ones((1, 1, 16)), torch.ones((1, 1, 16)), 1.0)
    assert bool((out[:2] == 0).all()) and bool((out[2] == 1).all())
