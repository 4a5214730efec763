"""The serving operators at the edges of their ranges, on the GPU against the CPU
oracle."""
import math

import pytest

torch = pytest.importorskip("torch")

from oracle import serving_oracle as O  # noqa: E402
from test_serving_gpu import TYPES, U, World, gen, run_attention, same, say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(i8l):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return i8l


def contents(cache):
    return {n: getattr(cache, n).clone()
            for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")}


# ---- non-finite values in the incomplete page ---------------------------------------

HIDDEN = [
    # len, queries, H, G, D, P, window, distance of the bad token from the end
    (40, 30, 1, 1, 64, 64, 0, 3),           # 16 rows a workgroup
    (40, 9, 2, 3, 48, 64, 0, 3),
    (104, 30, 1, 1, 80, 64, 5, 20),          # behind the window of the last queries
    (100, 1, 2, 1, 64, 64, 5, 20),           # a single query, the bad token behind its window
    (227, 100, 1, 1, 128, 128, 0, 60),       # a tail of two tiles, the bad token in the first
    (227, 100, 1, 1, 256, 128, 9, 10),       # ... in the second
    (3000, 12, 1, 1, 64, 128, 0, 5),         # keys split over workgroups
    (2410, 300, 8, 4, 64, 128, 0, 7),        # runs: 256 rows a workgroup
    (1400, 1200, 8, 8, 80, 128, 40, 70),     # ... the bad token behind the window
    (1120, 300, 6, 3, 256, 64, 0, 9),        # runs: 128 rows a workgroup
    (7100, 40, 8, 2, 128, 128, 0, 11),       # ... split
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,m,H,G,D,P,window,back", HIDDEN)
def test_attention_tail_hides_non_finite_values(lib, n, m, H, G, D, P, window, back, dtype):
    """An infinity or a NaN in a token of the incomplete page shows in the queries that
    see the token, in its dimension and sign, and in no other."""
    say("hidden values", n, m, H, G, D, P, window, back, dtype)
    w = World(lib, [n], H, D, P, dtype, seed=n + m + D, fill=False)
    bad = n - 1 - back
    assert bad >= n // P * P
    clean = w.v[0].clone()
    w.v[0][bad, :, 1], w.v[0][bad, :, 2], w.v[0][bad, 0, 3] = math.inf, -math.inf, math.nan
    w.write([0], [n])
    q = torch.randn((m, H * G, D), generator=gen(n)).to(w.dt)
    y = lib.cache_attention(q.cuda(), w.cache, w.table, w.lengths, cu=w.cu([m]), slots=w.slots,
                            window=window).cpu().double()
    pos = torch.arange(n - m, n)
    sees = pos >= bad
    if window:
        sees &= pos - bad < window
    w.v[0] = clean
    (k, v, s), = w.stored()
    o, tol = O.attention(q, k, v, D ** -0.5, window, None, s, U[w.dt])
    good = (y - o).abs() <= tol
    assert bool(good[~sees].all())
    assert bool(good[sees][:, :, 4:].all()) and bool(good[sees][:, :, 0].all())
    assert bool((y[sees][:, :, 1] == math.inf).all()) and bool((y[sees][:, :, 2] == -math.inf).all())
    assert bool(y[sees][:, :G, 3].isnan().all()) and bool(good[sees][:, G:, 3].all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,m,H,G,D,P,window,back", HIDDEN)
def test_attention_tail_hides_non_finite_keys(lib, n, m, H, G, D, P, window, back, dtype):
    """A key of NaNs in the incomplete page: the queries that see it are NaN, the others
    are as without it."""
    say("hidden keys", n, m, H, G, D, P, window, back, dtype)
    w = World(lib, [n], H, D, P, dtype, seed=n + m + D, fill=False)
    bad = n - 1 - back
    clean = w.k[0].clone()
    w.k[0][bad] = math.nan
    w.write([0], [n])
    q = torch.randn((m, H * G, D), generator=gen(n)).to(w.dt)
    y = lib.cache_attention(q.cuda(), w.cache, w.table, w.lengths, cu=w.cu([m]), slots=w.slots,
                            window=window).cpu().double()
    pos = torch.arange(n - m, n)
    sees = pos >= bad
    if window:
        sees &= pos - bad < window
    w.k[0] = clean
    (k, v, s), = w.stored()
    o, tol = O.attention(q, k, v, D ** -0.5, window, None, s, U[w.dt])
    assert bool(((y - o).abs() <= tol)[~sees].all())
    assert bool(y[sees].isnan().all())


def test_attention_infinity_far_below_the_maximum(lib):
    """An infinite value whose weight is below fp32's range, in a split of its own or not:
    the output is not finite (its weight is positive)."""
    for n in (300, 5000):
        w = World(lib, [n], 1, 64, 128, "fp16", seed=n, fill=False)
        w.v[0][n - 1, 0, 3] = math.inf
        w.k[0][:100] = 30.0
        w.k[0][n - 1] = -30.0
        w.write([0], [n])
        q = torch.ones((1, 1, 64)).half().cuda()
        y = lib.cache_attention(q, w.cache, w.table, w.lengths, slots=w.slots).cpu()[0, 0]
        assert not bool(y[3].isfinite())
        assert bool(y[:3].isfinite().all()) and bool(y[4:].isfinite().all())


# ---- the norm over bf16's range -----------------------------------------------------


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("K", [256, 1040, 4096, 14336, 40000, 65552])
def test_rmsnorm_quant_over_the_range_of_bf16(lib, K, eps):
    """Rows whose squares fp32 cannot hold, at both ends: the scale is absmax / rms there
    as anywhere, for every launch shape and with h in place of either operand."""
    say("rmsnorm_quant over bf16's range", K, eps)
    E = [126, 120, 100, 70, 64, 60, 0, -40, -60, -66, -70, -75, -80, -90]
    g = gen(K)
    base = (torch.rand((len(E), K), generator=g) * 1.5 - 0.75).bfloat16()
    base[:, 3] = 1.0
    two = torch.tensor([2.0 ** e for e in E])[:, None]
    X = (base.float() * two).bfloat16()        # (powers of two: exact)
    X[0, 5] = 1.0                              # one small value in a row of huge ones
    R = (X.float() * 0.25).bfloat16()
    W = (1 + 0.1 * torch.rand(K, generator=g)).bfloat16()
    for r, w in ((None, None), (R, W)):
        x, rr = X.cuda(), None if r is None else r.cuda()
        q0, s0, h0 = O.rmsnorm_quant(X, w, r, eps)
        q, s, h = lib.rmsnorm_quant(x, None if w is None else w.cuda(), residual=rr, eps=eps)
        same(q, q0)
        same(h, h0)
        # the tolerance of test_rmsnorm_quant, and fp32's last place where the scale is
        # below its normal numbers
        assert bool(((s.cpu().double() - s0).abs() <= 1e-5 * s0 + 2.0 ** -149).all())
        if r is not None:
            q2, s2, h2 = lib.rmsnorm_quant(x, w.cuda(), residual=rr, eps=eps, residual_out=rr)
            same(q2, q0)
            same(h2, h0)
            same(s2, s)


def test_rmsnorm_quant_small_weights_and_large_eps(lib):
    """Rows of subnormals lifted by their weight, an eps near fp32's largest: the scale is
    a / sqrt(mean h^2 + eps)."""
    X = torch.rand((3, 512), generator=gen(1)) * 0.5
    X[:, 1] = 1.0
    X = (X * torch.tensor([2.0 ** -120, 2.0 ** 63, 2.0 ** 80])[:, None]).bfloat16()
    W = torch.full((512,), 2.0 ** 40).bfloat16()
    W[7] = 2.0 ** 20
    for w, eps in ((W, 0.0), (W, 1e-30), (None, 3e38), (W * 2.0 ** -60, 1e38)):
        q0, s0, _ = O.rmsnorm_quant(X, w, None, eps)
        q, s, _ = lib.rmsnorm_quant(X.cuda(), None if w is None else w.cuda(), eps=eps)
        same(q, q0)
        s = s.cpu().double()
        assert bool(((s - s0).abs() <= 1e-5 * s0 + 2.0 ** -149).all()), (eps, s, s0)


def test_rmsnorm_quant_non_finite_rows_of_bf16(lib):
    """An infinity or a NaN in h still shows in the scale of its row, beside rows of huge
    finite values."""
    X = (torch.rand((5, 1040), generator=gen(2)) + 0.5).bfloat16() * 2.0 ** 100
    X[1, 700], X[3, 2] = math.inf, math.nan
    R = X.clone()
    R[4, 9] = X[4, 9] = 3.0e38                 # their sum overflows
    _, s, h = lib.rmsnorm_quant(X.cuda(), residual=R.cuda())
    s = s.cpu()
    assert s.isnan().tolist() == [False, True, False, True, True]
    assert bool((s[[0, 2]] > 0).all()) and bool(s[[0, 2]].isfinite().all())


# ---- sequences that outgrow their page table ------------------------------------------


def test_cache_write_past_the_page_table(lib):
    """Tokens past max_pages * page_size are skipped: complete pages and tails keep their
    bits, whatever the slot holds by then; the tokens before the end are written."""
    P, H, D = 16, 2, 64
    w = World(lib, [32, 30, 20], H, D, P, "fp16", seed=31)
    w.cache.k_tail[int(w.slots[0])] = 3.0          # sequence 0 has no tail: its slot is anyone's
    w.cache.v_tail[int(w.slots[0])] = 3.0
    before = contents(w.cache)
    k = torch.randn((3, H, D), generator=gen(1)).half().cuda()
    lens = torch.tensor([33, 40, 1 << 30], dtype=torch.int32, device="cuda")
    lib.cache_write(w.cache, k, k, w.table, lens, slots=w.slots)
    for name, t in contents(w.cache).items():
        same(t, before[name])
    # six new tokens of sequence 1, two of which its table holds
    new_k, new_v = (torch.randn((6, H, D), generator=gen(s)).half() for s in (2, 3))
    table = w.table[1:2].contiguous()
    lib.cache_write(w.cache, new_k.cuda(), new_v.cuda(), table,
                    torch.tensor([36], dtype=torch.int32, device="cuda"), cu=w.cu([6]),
                    slots=w.slots[1:2].contiguous())
    w.k[1], w.v[1] = torch.cat([w.k[1], new_k[:2]]), torch.cat([w.v[1], new_v[:2]])
    w.lens = [32, 32, 20]
    w.check_content()


@pytest.mark.parametrize("m,H,G", [(1, 2, 2), (3, 2, 2), (300, 8, 4)])
def test_attention_past_the_page_table(lib, m, H, G):
    """The positions of queries count the tokens past the table, which are out of sight."""
    P, D, held, n, window = 64, 64, 1024, 1027, 300
    w = World(lib, [held], H, D, P, "fp16", seed=32)
    q = torch.randn((m, H * G, D), generator=gen(m)).half()
    y = lib.cache_attention(q.cuda(), w.cache, w.table,
                            torch.tensor([n], dtype=torch.int32, device="cuda"), cu=w.cu([m]),
                            slots=w.slots, window=window).cpu().double()
    (k, v, s), = w.stored()
    for j in range(m):
        last = min(n - m + j, held - 1)
        first = max(0, n - m + j + 1 - window)
        if j % 37 and 2 < j < m - 4:
            continue
        # the last query of a sequence that ends at `last`, over the keys from `first` on
        o, tol = O.attention(q[j:j + 1], k[first:last + 1], v[first:last + 1], D ** -0.5,
                             page_scale=s[first:last + 1])
        assert bool(((y[j:j + 1] - o).abs() <= tol).all()), j


# ---- pages and slots outside the cache --------------------------------------------------


def test_cache_write_outside_the_cache_touches_nothing_else(lib):
    """With page numbers and slots outside the cache every other byte keeps its value: all
    six tensors."""
    w = World(lib, [48, 20], 1, 64, 16, "fp16", seed=4)
    before = contents(w.cache)
    table = w.table.clone()
    table[0, :3] = torch.tensor([-5, w.cache.n_pages, 2 ** 31 - 1])
    slots = torch.tensor([-1, 99], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((68, 1, 64), generator=gen(s)).half() for s in (5, 6))
    lib.cache_write(w.cache, k.cuda(), v.cuda(), table, w.lengths, cu=w.cu([48, 20]), slots=slots)
    p, st = int(table[1, 0]), O.Store(16)
    for name, x, tr in (("k", k, False), ("v", v, True)):
        c, s = st.page(x[48:64, 0])
        want = before[name + "_codes"]
        want[p, 0] = (c.t() if tr else c).to(want.device)
        same(getattr(w.cache, name + "_codes"), want)
        want = before[name + "_scale"]
        want[p, 0] = s
        same(getattr(w.cache, name + "_scale"), want)
        same(getattr(w.cache, name + "_tail"), before[name + "_tail"])


def test_slots_outside_the_cache_hide_the_tail(lib):
    """Attention masks the tokens of a slot outside the cache, in both kernels; cache_read
    gives zeros for them."""
    lens, H, G, D, P = [1000, 20], 8, 2, 64, 64
    w = World(lib, lens, H, D, P, "fp16", seed=41)
    for slots in ([-1, 99], [2 ** 31 - 1, -2 ** 31]):
        slots = torch.tensor(slots, dtype=torch.int32, device="cuda")
        for m in (1, 200, 600):
            Q = [m, min(m, 20)]
            q = [torch.randn((c, H * G, D), generator=gen(c)).half() for c in Q]
            y = lib.cache_attention(torch.cat(q).cuda(), w.cache, w.table, w.lengths, cu=w.cu(Q),
                                    slots=slots).cpu().double()
            assert bool((y[m:] == 0).all())
            k, v, s = w.stored()[0]
            held = 1000 // P * P
            j = min(m, held - (1000 - m))          # rows whose token is in a complete page
            if j > 0:
                o, tol = O.attention(q[0][:j], k[:1000 - m + j], v[:1000 - m + j], D ** -0.5,
                                     page_scale=s[:1000 - m + j])
                assert bool(((y[:j] - o).abs() <= tol).all())
            o, tol = O.attention(q[0][-1:], k[:held], v[:held], D ** -0.5, page_scale=s[:held])
            assert bool(((y[m - 1:m] - o).abs() <= tol).all())
        k, v = lib.cache_read(w.cache, w.table, w.lengths, w.cu(lens), 1020, slots=slots)
        for got, i in ((k, 0), (v, 1)):
            same(got[:held], w.stored()[0][i][:held].half())
            assert bool((got[held:] == 0).all())


# ---- workspaces that the caller gives, or does not ---------------------------------------


@pytest.mark.parametrize("M,K,N", [(1, 4096, 1000), (8, 4096, 16384), (65, 2064, 257), (300, 8208, 1000),
                                   (300, 8208, 2000), (520, 8208, 1900), (200, 1040, 16500),
                                   (512, 2048, 33000)])
def test_linear_codes_workspaces(lib, M, K, N):
    """The caller's workspace, one too large, and none at all (nothing is then split along
    k) give the same bits; one too small is refused."""
    from mixed_precision_quantized_int8_amd._binding import check

    say("linear_codes, workspaces", M, K, N)
    g = gen(M + N)
    Xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8).cuda()
    Wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sx, sw = torch.rand(M, generator=g).cuda(), (torch.rand(N, generator=g) * 0.1).cuda()
    y0, mag = O.linear_codes(Xq.cpu(), sx.cpu(), Wq.cpu(), sw.cpu())
    want = lib.linear_codes(Xq, sx, Wq, sw)
    # the tolerance of test_linear_codes
    assert bool(((want.cpu().double() - y0).abs()
                 <= 2.0 ** -11 * y0.abs() + 2.0 ** -22 * mag + 2.0 ** -25).all())
    need = lib.lib().i8l_codes_workspace_bytes(M, K, N)
    for extra in (0, 4096):
        ws = torch.full((need + extra,), 0x7f, dtype=torch.uint8, device="cuda")
        same(lib.linear_codes(Xq, sx, Wq, sw, workspace=ws), want)
    out = torch.full_like(want, math.nan)
    check(lib.lib().int8_linear_codes(Xq.data_ptr(), sx.data_ptr(), M, K, Wq.data_ptr(), sw.data_ptr(),
                                      N, None, out.data_ptr(), None, 0,
                                      torch.cuda.current_stream().cuda_stream))
    same(out, want)
    if need > 16:
        with pytest.raises(lib.Int8LinError, match="workspace"):
            lib.linear_codes(Xq, sx, Wq, sw, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_attention_workspaces(lib):
    """The caller's workspace holds the partial results; a call without one allocates it."""
    w = World(lib, [3000, 700], 2, 64, 64, "fp16", seed=51)
    q = torch.randn((2, 4, 64), generator=gen(7)).half().cuda()
    args = (q, w.cache, w.table, w.lengths)
    want = lib.cache_attention(*args, slots=w.slots, max_len=3000)
    need = lib.attention_workspace_bytes(w.cache, 2, 4, 1, 3000)
    assert need > 0
    for extra in (0, 1 << 16):
        ws = torch.full((need + extra,), 0x7f, dtype=torch.uint8, device="cuda")
        same(lib.cache_attention(*args, slots=w.slots, max_len=3000, workspace=ws), want)
    with pytest.raises(lib.Int8LinError, match="workspace"):
        lib.cache_attention(*args, slots=w.slots, max_len=3000, workspace=ws[:need - 16])


# ---- a cache and its tensors ----------------------------------------------------------


def test_a_larger_pool_is_a_new_cache(lib):
    """A cache's tensors stay as they were made; the pages of one move into a larger one
    by copying the tensors."""
    w = World(lib, [40, 33], 2, 64, 16, "fp16", seed=61)
    with pytest.raises(AttributeError, match="new one"):
        w.cache.k_codes = torch.empty_like(w.cache.k_codes)
    old = w.cache
    big = lib.new_cache(old.n_pages + 5, old.n_slots, 2, 64, 16, w.dt, "cuda:0")
    for name, t in contents(old).items():
        getattr(big, name)[:t.shape[0]].copy_(t)
    w.cache = big
    w.check_content()
    run_attention(w, 2, [1, 1])


# ---- partial results of split keys --------------------------------------------------------


@pytest.mark.parametrize("lens,Q,H,G,D,alibi", [
    ([700], 1, 1, 1, 64, False), ([700, 650, 600], 1, 5, 1, 80, True), ([700], 1, 1, 1, 256, False),
    ([2000, 30], 1, 1, 7, 176, False), ([900], 3, 1, 1, 128, False), ([2800], 33, 3, 1, 256, True)])
def test_attention_odd_numbers_of_partial_results(lib, lens, Q, H, G, D, alibi):
    """Rows times splits odd, and heads of 256 with split keys."""
    for dtype in TYPES:
        say("odd partial results", lens, Q, H, G, D, alibi, dtype)
        w = World(lib, lens, H, D, 32, dtype, seed=sum(lens) + D)
        assert lib.attention_workspace_bytes(w.cache, len(lens), H * G, Q, max(lens)) > 0
        run_attention(w, G, [Q] * len(lens), 0, alibi)
