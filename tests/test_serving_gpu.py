"""The serving operators on the GPU against the CPU oracle: row norm to codes,
product of codes, the 8-bit key/value cache (written, read back) and attention
over it.

Codes, page scales and tails are bit-exact; sx, Y and attention outputs are held
to tolerances derived from the arithmetic (stated where they are used).
"""
import math

import pytest

torch = pytest.importorskip("torch")

from oracle import serving_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def lib(i8l):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return i8l


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def same(a, b):
    """Equal bit for bit (NaN with NaN)."""
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    eq = a == b
    if a.is_floating_point():
        eq |= a.isnan() & b.isnan()
    assert bool(eq.all()), f"{int((~eq).sum())} of {eq.numel()} differ"


# ---- norm -----------------------------------------------------------------------

# one case per launch shape, odd row counts, the largest K
NORM = [(1, 16), (5, 512), (4, 528), (3, 1024), (2, 1040), (3, 2048), (1, 4096), (7, 4112), (2, 8192), (3, 14336),
        (2, 16400), (1, 32784), (1, 57344), (2, 65552), (1, 133136), (300, 256), (1000, 1040)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", NORM)
def test_rmsnorm_quant(lib, M, K, dtype):
    say("rmsnorm_quant", M, K, dtype)
    dt, g = TYPES[dtype], gen(M * 7 + K)
    X = torch.randn((M, K), generator=g).to(dt)
    R = (3 * torch.randn((M, K), generator=g)).to(dt)
    W = (1 + 0.3 * torch.randn(K, generator=g)).to(dt)
    if M > 2:
        X[1] = 0
        R[1] = 0          # a zero row: scale 0, codes 0
    for res, w, eps in ((R, W, 1e-5), (None, W, 0.25), (R, None, 1e-6), (None, None, 1e-5)):
        q, s, h = lib.rmsnorm_quant(X.cuda(), None if w is None else w.cuda(),
                                    residual=None if res is None else res.cuda(), eps=eps)
        q0, s0, h0 = O.rmsnorm_quant(X, w, res, eps)
        same(q, q0)
        same(h, h0)
        # at most 8 * 17 + 6 + 16 additions on a path, then a division, a root, a
        # division: below 161 + 3 roundings of 2^-24, halved by the root
        assert bool(((s.cpu().double() - s0).abs() <= 1e-5 * s0).all())


def test_rmsnorm_quant_ties_and_in_place(lib):
    """Codes at exact ties go away from zero; the residual may be written in place."""
    X = torch.zeros((2, 64), dtype=torch.float16)
    X[0, :8] = torch.tensor([127.0, 0.5, -0.5, 1.5, -1.5, 2.5, 126.5, -126.5])
    X[1] = X[0] * 2
    q, s, h = lib.rmsnorm_quant(X.cuda())
    want = torch.tensor([127, 1, -1, 2, -2, 3, 127, -127], dtype=torch.int8)
    same(q[0, :8], want)
    same(q[1, :8], want)
    R = torch.ones((2, 64), dtype=torch.float16, device="cuda")
    q2, s2, h2 = lib.rmsnorm_quant(X.cuda(), residual=R, residual_out=R)
    assert h2.data_ptr() == R.data_ptr()
    same(R, X + 1)
    same(q2, O.rmsnorm_quant(X + 1)[0])


@pytest.mark.parametrize("K", [64, 4096, 57344, 65552])
def test_rmsnorm_quant_writes_h_over_its_inputs(lib, K):
    """h over the residual, and over X: the same codes and scales as into a tensor of
    its own (the widest rows are read twice)."""
    g = gen(K)
    X, R = (torch.randn((3, K), generator=g).half().cuda() for _ in range(2))
    W = (1 + 0.2 * torch.randn(K, generator=g)).half().cuda()
    q, s, h = lib.rmsnorm_quant(X, W, residual=R)
    for over in ("residual", "X"):
        x, r = X.clone(), R.clone()
        out = r if over == "residual" else x
        q2, s2, h2 = lib.rmsnorm_quant(x, W, residual=r, residual_out=out)
        assert h2.data_ptr() == out.data_ptr()
        same(h2, h)
        same(q2, q)
        same(s2, s)


def test_rmsnorm_quant_non_finite_rows(lib):
    """A NaN or an infinity shows in its own row's scale and in no other."""
    X = torch.randn((4, 256), generator=gen(1)).half()
    clean = lib.rmsnorm_quant(X.cuda())
    X[1, 3], X[2, 200] = math.nan, math.inf
    q, s, h = lib.rmsnorm_quant(X.cuda())
    assert bool(s[1].isnan()) and bool(s[2].isnan())
    for i in (0, 3):
        same(q[i], clean[0][i])
        same(s[i], clean[1][i])


@pytest.mark.parametrize("K", [256, 4096, 65552])
def test_rmsnorm_quant_non_finite_weight(lib, K):
    """A NaN in the weight shows in every row's scale, an infinity too."""
    X = torch.rand((3, K), generator=gen(K)).half() + 1
    for bad in (math.nan, math.inf, -math.inf):
        W = torch.ones(K).half()
        W[K - 5] = bad
        _, s, h = lib.rmsnorm_quant(X.cuda(), W.cuda())
        same(h, X)
        assert not bool(s.isfinite().any())
        assert bool(s.isnan().all()) or not math.isnan(bad)


def test_rmsnorm_quant_very_small_rows(lib):
    """bf16 rows over the small end of the type's range: below 2^-93 codes and scale 0;
    a zero among them is code 0 everywhere, also with eps = 0."""
    X = torch.rand((6, 512), generator=gen(8)) * 2 - 1
    X[:, 5], X[:, 9] = 1.0, 0.0
    X = X.bfloat16()
    W = torch.ones(512)
    X[4] = 0
    for i, e in enumerate((-126, -120, -94, -92)):   # (powers of two: exact)
        W2 = (W * 2.0 ** (e // 2)).bfloat16()
        Y = X.clone()
        Y[:4] = Y[:4] * 2.0 ** (e - e // 2)
        for eps in (0.0, 1e-5):
            q, s, h = lib.rmsnorm_quant(Y.cuda(), W2.cuda(), eps=eps)
            q0, s0, _ = O.rmsnorm_quant(Y, W2, None, eps)
            same(q, q0)
            # squares of rows near 2^-63 are fp32 subnormals, and the row's own eps-free
            # root with them: the scale is held to eps > 0, and zeros to both
            assert bool((s.cpu()[s0 == 0] == 0).all())
            if eps:
                assert bool(((s.cpu().double() - s0).abs() <= 1e-5 * s0 + 2.0 ** -126).all())


# ---- product --------------------------------------------------------------------

CODES = [(1, 16, 1), (1, 4096, 1000), (8, 4096, 16384), (16, 1024, 33), (17, 272, 130), (64, 2064, 1300),
         (65, 528, 257), (128, 1040, 64), (129, 1024, 300), (256, 4096, 515), (257, 80, 300), (520, 2048, 1300),
         (700, 1040, 77)]
# the layer's own kernels on codes: streaming, skinny tiles, 256 x 256 tiles whole and split
CODES += [(32, 1040, 5000), (3, 528, 8500), (80, 272, 16400), (200, 1040, 16500), (300, 80, 16640), (512, 2048, 33000)]
# 128 features a tile: many tiles, one of 32 features at the end, k split by 5
CODES += [(2300, 272, 1000), (1100, 1040, 2900), (300, 8208, 2050)]


@pytest.mark.parametrize("M,K,N", CODES)
def test_linear_codes(lib, M, K, N):
    say("linear_codes", M, K, N)
    g = gen(M + K + N)
    Xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    Wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g) * 5, torch.rand(N, generator=g) * 0.1
    sx[0] = 0
    bias = torch.randn(N, generator=g).half()
    for b in (None, bias):
        y0, mag = O.linear_codes(Xq, sx, Wq, sw, b)
        # one fp16 rounding; int32 -> fp32, two scale products, the sum: 4 roundings of 2^-24
        tol = 2.0 ** -11 * y0.abs() + 2.0 ** -22 * mag + 2.0 ** -25
        out = torch.full((M, N), math.nan, dtype=torch.float16, device="cuda")
        y = lib.linear_codes(Xq.cuda(), sx.cuda(), Wq.cuda(), sw.cuda(),
                             bias=None if b is None else b.cuda(), out=out)
        assert y.data_ptr() == out.data_ptr()
        assert bool(((y.cpu().double() - y0).abs() <= tol).all())
    again = lib.linear_codes(Xq.cuda(), sx.cuda(), Wq.cuda(), sw.cuda(), bias=bias.cuda())
    same(again, y)


def test_linear_codes_extreme_sums(lib):
    """The largest K with every product at its largest: the int32 sum is exact."""
    K, N = 133136, 48
    for M in (2, 70, 300):
        Xq = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
        Wq = torch.full((N, K), -127, dtype=torch.int8, device="cuda")
        one = torch.ones(max(M, N), device="cuda")
        y = lib.linear_codes(Xq, one[:M] * 2.0 ** -8, Wq, one[:N].clone())
        want = torch.full((M, N), -K * 2.0 ** -8).half()
        same(y, want)


def test_norm_then_codes_is_the_layer_without_outliers(lib):
    """With the norm's identity weight the pair matches the layer on the same rows:
    codes of x are codes of x / rms, scales differ by rms."""
    g = gen(5)
    X = torch.randn((40, 1024), generator=g).half().cuda()
    W = (torch.randn((1024, 264), generator=g) * 0.02).half().cuda()
    Wq, sw = lib.quantize_weight(W)
    o = lib.quantize_activation(X, 0.0)
    Xq, sx, h = lib.rmsnorm_quant(X, eps=0.0)
    same(Xq, o["Xq"])
    y = lib.linear_codes(o["Xq"], o["sx"], Wq, sw)
    same(y, lib.linear(X, Wq, sw, W, 0.0))


# ---- the cache ------------------------------------------------------------------


class World:
    """A cache of random contents with a page table, on the GPU, beside the 16-bit
    tokens that were written (CPU)."""

    def __init__(self, lib, lens, H, D, P, dtype, seed=0, spare=3, fill=True, scale=1.0):
        g = gen(seed)
        dt = TYPES[dtype]
        B, per = len(lens), max(1, -(-max(lens) // P))
        self.lib, self.lens, self.P, self.H, self.D, self.dt = lib, lens, P, H, D, dt
        n = B * per + spare
        self.cache = lib.new_cache(n, B + 2, H, D, P, dt, "cuda:0")
        # what was in the memory before: codes of anything, NaN scales and tails
        for t in (self.cache.k_scale, self.cache.v_scale, self.cache.k_tail, self.cache.v_tail):
            t.fill_(math.nan)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.fill_(77)
        order = torch.randperm(n, generator=g)[:B * per].view(B, per).to(torch.int32)
        for b, m in enumerate(lens):   # entries past a sequence's pages name no page
            order[b, -(-m // P):] = -1 if b % 2 else 1 << 30
        self.table = order.cuda()
        self.slots = torch.randperm(B + 2, generator=g)[:B].to(torch.int32).cuda()
        self.lengths = torch.tensor(lens, dtype=torch.int32).cuda()
        self.k = [(torch.randn((m, H, D), generator=g) * scale).to(dt) for m in lens]
        self.v = [(torch.randn((m, H, D), generator=g) * scale).to(dt) for m in lens]
        if fill:
            self.write([0] * B, lens)

    def cu(self, counts):
        return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32,
                            device="cuda")

    def write(self, lo, hi, **kw):
        """Writes tokens lo[b] .. hi[b] - 1 of every sequence in one call."""
        k = torch.cat([x[a:b] for x, a, b in zip(self.k, lo, hi)]).cuda()
        v = torch.cat([x[a:b] for x, a, b in zip(self.v, lo, hi)]).cuda()
        n = [b - a for a, b in zip(lo, hi)]
        self.lib.cache_write(self.cache, k, v, self.table,
                             torch.tensor(hi, dtype=torch.int32, device="cuda"), cu=self.cu(n),
                             slots=self.slots, **kw)

    def stored(self):
        """Per sequence: values (k, v) [n][H][D] fp32 and page scales per token of v."""
        out = []
        st = O.Store(self.P)
        for k, v in zip(self.k, self.v):
            kv, _ = st.sequence(k)
            vv, pages = st.sequence(v)
            s = torch.ones((len(v), self.H))
            for g, per in enumerate(pages):
                for h, (_, sc) in enumerate(per):
                    s[g * self.P:(g + 1) * self.P, h] = sc
            out.append((kv, vv, s))
        return out

    def check_content(self):
        """Codes, scales and tails of the cache, bit for bit."""
        st = O.Store(self.P)
        c = self.cache
        for b, (k, v) in enumerate(zip(self.k, self.v)):
            n = self.lens[b]
            full, slot = n // self.P, int(self.slots[b])
            for x, cc, ss, tt, tr in ((k, c.k_codes, c.k_scale, c.k_tail, False),
                                      (v, c.v_codes, c.v_scale, c.v_tail, True)):
                _, pages = st.sequence(x)
                for g in range(full):
                    page = int(self.table[b, g])
                    want = torch.stack([p[0].t() if tr else p[0] for p in pages[g]])
                    same(cc[page], want)
                    same(ss[page], torch.stack([p[1] for p in pages[g]]))
                r = n - full * self.P
                if r:
                    tail = tt[slot, :, :, :r].transpose(1, 2) if tr else tt[slot, :, :r]
                    same(tail.transpose(0, 1).contiguous(), x[full * self.P:])


CACHE = [
    # lens, H, D, P
    ([5], 1, 16, 16),
    ([16, 15, 17, 0, 1], 2, 64, 16),
    ([33, 64, 100], 3, 80, 32),
    ([64, 128, 200, 63], 2, 128, 64),
    ([300, 127, 128], 2, 128, 128),
    ([130, 7], 1, 256, 128),
    ([1000], 5, 96, 32),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,H,D,P", CACHE)
def test_cache_write_and_read(lib, lens, H, D, P, dtype):
    say("cache", lens, H, D, P, dtype)
    w = World(lib, lens, H, D, P, dtype, seed=sum(lens) + D)
    w.check_content()
    total = sum(lens)
    k, v = lib.cache_read(w.cache, w.table, w.lengths, w.cu(lens), total, slots=w.slots)
    for got, i in ((k, 0), (v, 1)):
        same(got, torch.cat([s[i].to(w.dt) for s in w.stored()]))


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_cache_content_does_not_depend_on_the_calls(lib, P, dtype):
    """Written at once, token by token, and in ragged chunks that start and end inside
    pages: the same codes, scales and tails."""
    say("cache split", P, dtype)
    lens = [P * 3 + 5, P * 2, 9]
    for cuts in ([1.0], None, [0.1, 0.33, 0.34, 0.8, 1.0]):
        w = World(lib, lens, 2, 64, P, dtype, seed=3, fill=False)
        at = [0, 0, 0]
        if cuts is None:
            steps = [[min(n, i + 1) for n in lens] for i in range(max(lens))]
        else:
            steps = [[int(round(n * c)) for n in lens] for c in cuts]
        for to in steps:
            w.write(at, to)
            at = to
        assert at == lens
        w.check_content()


def test_cache_one_token_form_and_strides(lib):
    """Without cu each row belongs to its sequence; rows may be views into a fused
    projection, in either order of heads and parts."""
    H, D, P, B = 4, 64, 16, 5
    lens = [16, 1, 17, 40, 32]
    w = World(lib, lens, H, D, P, "fp16", seed=9, fill=False)
    w.write([0] * B, [n - 1 for n in lens])
    fused = torch.full((B, H, 3, D), math.nan, dtype=torch.float16)
    for b in range(B):
        fused[b, :, 1], fused[b, :, 2] = w.k[b][-1], w.v[b][-1]
    f = fused.cuda()
    lib.cache_write(w.cache, f[:, :, 1], f[:, :, 2], w.table, w.lengths, slots=w.slots)
    w.check_content()


def test_cache_zero_and_non_finite_pages(lib):
    w = World(lib, [64, 40], 2, 64, 16, "fp16", seed=2, fill=False)
    w.k[0][16:32] = 0           # scale 0
    w.v[0][:16, 1] = 0
    w.k[1][3, 0, 5] = math.inf  # page 0 of head 0 reads as NaN, head 1 and page 1 do not
    w.v[1][20, 1, 7] = math.nan
    w.write([0, 0], w.lens)
    w.check_content()
    k, v = lib.cache_read(w.cache, w.table, w.lengths, w.cu(w.lens), 104, slots=w.slots)
    st = w.stored()
    same(k, torch.cat([s[0].half() for s in st]))
    same(v, torch.cat([s[1].half() for s in st]))
    assert bool(k[64:80, 0].isnan().all()) and not bool(k[64:80, 1].isnan().any())


@pytest.mark.parametrize("e", [-126, -120, -112, -105, -94, -93, -92, -60, 120])
def test_cache_pages_of_very_small_and_large_values(lib, e):
    """bf16 pages over the type's range: below 2^-93 zeros, from there on codes as
    anywhere (of 127 * 2^16 / absmax nothing overflows)."""
    w = World(lib, [48], 2, 32, 16, "bf16", seed=e + 200, fill=False)
    for x in (w.k[0], w.v[0]):
        x[16:32] = (torch.rand((16, 2, 32), generator=gen(5)) * 2 - 1).to(w.dt) * 2.0 ** e
        x[20, :, 3] = 2.0 ** e
    w.write([0], w.lens)
    w.check_content()
    k, v = lib.cache_read(w.cache, w.table, w.lengths, w.cu(w.lens), 48, slots=w.slots)
    (k0, v0, _), = w.stored()
    same(k, k0.to(w.dt))
    same(v, v0.to(w.dt))


def test_cache_ignores_pages_and_slots_outside(lib):
    """A table entry or slot outside the cache is skipped: nothing else changes."""
    w = World(lib, [48, 20], 1, 64, 16, "fp16", seed=4)
    before = [t.clone() for t in (w.cache.k_codes, w.cache.v_codes)]
    table = w.table.clone()
    table[0, :3] = torch.tensor([-5, w.cache.n_pages, 2 ** 31 - 1])
    slots = torch.tensor([-1, 99], dtype=torch.int32, device="cuda")
    k = torch.randn((68, 1, 64)).half().cuda()
    lens = torch.tensor([48, 20], dtype=torch.int32, device="cuda")
    lib.cache_write(w.cache, k, k, table, lens, cu=w.cu([48, 20]), slots=slots)
    # sequence 1's one complete page is the only one that may differ
    p = int(table[1, 0])
    for old, now in zip(before, (w.cache.k_codes, w.cache.v_codes)):
        d = (old != now).flatten(1).any(1)
        assert d.nonzero().flatten().tolist() in ([], [p])


# ---- attention ------------------------------------------------------------------


def run_attention(w, G, Q, window=0, alibi=False, seed=1, q_scale=1.0, **kw):
    """Queries of the last Q[b] tokens of every sequence, against the oracle."""
    lib, g = w.lib, gen(seed + 100)
    Hq = w.H * G
    q = [(torch.randn((m, Hq, w.D), generator=g) * q_scale).to(w.dt) for m in Q]
    slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / Hq) for i in range(Hq)]) if alibi else None
    one = all(m == 1 for m in Q)
    rows = torch.cat(q).cuda()
    out = torch.full(rows.shape, math.nan, dtype=w.dt, device="cuda")
    y = lib.cache_attention(rows, w.cache, w.table, w.lengths, cu=None if one else w.cu(Q),
                            slots=w.slots, window=window, out=out,
                            alibi=None if slopes is None else slopes.cuda(), **kw)
    y = y.cpu().double()
    assert not bool(y.isnan().any())
    at = 0
    for b, (k, v, s) in enumerate(w.stored()):
        o, tol = O.attention(q[b], k, v, kw.get("scale", w.D ** -0.5), window, slopes, s, U[w.dt])
        d = (y[at:at + Q[b]] - o).abs()
        assert bool((d <= tol).all()), f"sequence {b}: {float((d / tol).max()):.3g} of the tolerance"
        at += Q[b]


SINGLE = [
    # lens, H, G, D, P, window, alibi
    ([1], 1, 1, 16, 16, 0, False),
    ([1, 0, 15, 16, 17, 31, 64, 65], 2, 1, 64, 16, 0, False),
    ([100, 63, 129], 2, 4, 128, 64, 0, True),
    ([300, 256, 127, 128], 1, 8, 128, 128, 0, False),
    ([777, 30], 2, 3, 80, 32, 0, False),
    ([777, 30, 150], 2, 3, 80, 32, 100, True),
    ([400, 5, 33], 1, 1, 256, 16, 7, False),
    ([2000], 1, 16, 64, 16, 0, False),
    ([1500, 900], 1, 20, 64, 64, 0, False),
    ([5000], 1, 2, 128, 64, 0, True),
    ([3000], 2, 2, 96, 128, 1000, False),
    ([100, 64], 2, 2, 16, 16, 0, False),
    ([300], 1, 3, 32, 32, 0, True),
    ([257, 130], 2, 1, 48, 128, 0, False),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,H,G,D,P,window,alibi", SINGLE)
def test_attention_single_queries(lib, lens, H, G, D, P, window, alibi, dtype):
    say("attention, one query each", lens, H, G, D, P, window, alibi, dtype)
    w = World(lib, lens, H, D, P, dtype, seed=sum(lens) + G)
    run_attention(w, G, [1] * len(lens), window, alibi)


RUNS = [
    # lens, queries, H, G, D, P, window, alibi
    ([40], [40], 1, 1, 64, 16, 0, False),
    ([70, 33, 16], [3, 33, 1], 2, 2, 64, 16, 0, False),
    ([200, 150], [130, 7], 1, 3, 80, 32, 0, True),
    ([300], [257], 1, 1, 128, 64, 0, False),
    ([333, 333], [100, 333], 1, 2, 128, 128, 50, False),
    ([500, 0, 128], [64, 0, 128], 2, 1, 64, 64, 0, False),
    ([260], [130], 1, 2, 256, 16, 33, True),
    ([1200], [20], 1, 5, 128, 32, 0, False),
    ([1100], [300], 1, 1, 96, 16, 256, False),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,Q,H,G,D,P,window,alibi", RUNS)
def test_attention_runs_of_queries(lib, lens, Q, H, G, D, P, window, alibi, dtype):
    say("attention, runs", lens, Q, H, G, D, P, window, alibi, dtype)
    w = World(lib, lens, H, D, P, dtype, seed=sum(lens) + sum(Q))
    run_attention(w, G, Q, window, alibi)


# sizes that take the kernel for runs of queries: 128 and 256 rows a workgroup, whole
# and split, both padded head sizes, every page size, tails of one and two tiles
WIDE_RUNS = [
    # lens, queries, H, G, D, P, window, alibi
    ([1100, 333], [300, 290], 4, 4, 64, 16, 0, False),
    ([1100, 333], [300, 290], 4, 4, 128, 64, 0, True),
    ([7000], [40], 8, 2, 128, 128, 0, False),           # 80 rows, split
    ([5000, 100], [33, 100], 8, 2, 80, 32, 0, True),
    ([2303], [129], 16, 1, 96, 128, 0, False),           # 129 rows: 256 a workgroup; tail 127
    ([2800, 0, 2750], [520, 0, 300], 8, 3, 64, 64, 500, False),
    ([1100], [512], 48, 4, 64, 16, 70, True),
    ([1300, 1281], [513, 7], 8, 1, 128, 128, 1000, False),
    ([4500], [2100], 2, 1, 112, 32, 0, False),
    ([1025, 640, 511], [1025, 640, 400], 3, 2, 64, 128, 0, False),
    ([2100], [2100], 32, 1, 64, 64, 0, False),           # 256 rows a workgroup, not split
    ([1100, 1040], [400, 333], 6, 3, 16, 16, 0, False),
    ([1100, 1040], [400, 333], 6, 3, 256, 64, 0, False),
    ([2303], [129], 16, 1, 176, 128, 0, True),
    ([1100, 1040], [400, 333], 6, 3, 48, 64, 0, True),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,Q,H,G,D,P,window,alibi", WIDE_RUNS)
def test_attention_wide_runs(lib, lens, Q, H, G, D, P, window, alibi, dtype):
    say("attention, wide runs", lens, Q, H, G, D, P, window, alibi, dtype)
    w = World(lib, lens, H, D, P, dtype, seed=sum(lens) + sum(Q))
    run_attention(w, G, Q, window, alibi)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_wide_runs_extreme_values(lib, dtype):
    """As test_attention_extreme_values, through the kernel for runs: maxima that rise
    late and by much, value scales of many orders, pages of zeros."""
    w = World(lib, [1200, 700], 8, 64, 32, dtype, seed=18, fill=False)
    w.v[0][:256] *= 2.0 ** -10
    w.v[0][256:384] *= 512
    w.v[0][512:576] = 0
    w.k[0][576:640] = 0
    w.k[0][640:] *= 20           # scores that leave the first ones far behind
    w.k[1] *= 30
    w.write([0, 0], w.lens)
    run_attention(w, 2, [300, 300], q_scale=4.0)
    run_attention(w, 2, [300, 700], window=900)


def test_attention_wide_runs_hide_non_finite_pages(lib):
    """A page of NaNs shows in the rows that see it and in no other, in both kernels'
    masked tiles; a page number outside the cache hides its tokens."""
    H, n, m = 8, 1280, 1000
    w = World(lib, [n], H, 64, 16, "fp16", seed=19, fill=False)
    clean = [x.clone() for x in (w.k[0], w.v[0])]
    w.v[0][400, :, 1] = math.nan      # the page of tokens 400 .. 415
    w.write([0], w.lens)
    q = torch.randn((m, 2 * H, 64), generator=gen(2)).half()
    y = lib.cache_attention(q.cuda(), w.cache, w.table, w.lengths, cu=w.cu([m]), slots=w.slots)
    y = y.cpu().double()
    first = 400 - (n - m)             # the first query that sees token 400 of the page
    assert bool(y[first:].isnan().all())
    st = O.Store(16)
    k, (v, pages) = st.sequence(clean[0])[0], st.sequence(clean[1])
    s = torch.ones((n, H))
    for g, per in enumerate(pages):
        for h in range(H):
            s[g * 16:(g + 1) * 16, h] = per[h][1]
    o, tol = O.attention(q[:first], k[:400], v[:400], 64 ** -0.5, page_scale=s[:400])
    assert bool(((y[:first] - o).abs() <= tol).all())
    # the page's number replaced: its tokens are out of sight, for all rows
    table = w.table.clone()
    table[0, 25] = -7
    y = lib.cache_attention(q.cuda(), w.cache, table, w.lengths, cu=w.cu([m]), slots=w.slots)
    keep = torch.cat([torch.arange(400), torch.arange(416, n)])
    late = 416 - (n - m)
    o, tol = O.attention(q[late:], k[keep], v[keep], 64 ** -0.5, page_scale=s[keep])
    assert bool(((y[late:].cpu().double() - o).abs() <= tol).all())


def test_attention_rows_that_see_nothing(lib):
    """More rows than tokens: the first queries come before the sequence's first
    token and give 0; so does every query of an empty sequence."""
    w = World(lib, [3, 0, 20], 1, 64, 16, "fp16", seed=6)
    q = torch.randn((5 + 2 + 1, 2, 64), generator=gen(0)).half()
    y = lib.cache_attention(q.cuda(), w.cache, w.table, w.lengths, cu=w.cu([5, 2, 1]), slots=w.slots)
    y = y.cpu()
    assert bool((y[:2] == 0).all()) and bool((y[5:7] == 0).all())
    k, v, s = w.stored()[0]
    o, tol = O.attention(q[2:5], k, v, 64 ** -0.5, page_scale=s)
    assert bool(((y[2:5].double() - o).abs() <= tol).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_extreme_values(lib, dtype):
    """Scores far apart (one key takes all), pages of zeros, pages whose value scales
    differ by many orders: the small ones still count where they alone are seen."""
    w = World(lib, [200, 90], 2, 64, 16, dtype, seed=8, fill=False)
    w.v[0][:64] *= 2.0 ** -10
    w.v[0][64:96] *= 512
    w.v[0][112:128] = 0
    w.k[0][128:144] = 0
    w.k[1] *= 30
    w.write([0, 0], w.lens)
    run_attention(w, 2, [1, 1], q_scale=4.0)
    run_attention(w, 2, [1, 1], window=80)
    run_attention(w, 1, [200, 90])


def test_attention_non_finite_pages_stay_hidden(lib):
    """A page that reads as NaN shows in the queries that see it and in no other."""
    w = World(lib, [64], 1, 64, 16, "fp16", seed=10, fill=False)
    clean = [x.clone() for x in (w.k[0], w.v[0])]
    w.v[0][40, 0, 1] = math.nan      # page 2: tokens 32 .. 47
    w.write([0], w.lens)
    q = torch.randn((64, 1, 64), generator=gen(2)).half()
    y = lib.cache_attention(q.cuda(), w.cache, w.table, w.lengths, cu=w.cu([64]), slots=w.slots)
    y = y.cpu().double()
    assert bool(y[32:].isnan().all())
    st = O.Store(16)
    k, (v, pages) = st.sequence(clean[0])[0], st.sequence(clean[1])
    s = torch.ones((64, 1))
    for g, per in enumerate(pages):
        s[g * 16:(g + 1) * 16, 0] = per[0][1]
    o, tol = O.attention(q[:32], k[:32], v[:32], 64 ** -0.5, page_scale=s[:32])
    assert bool(((y[:32] - o).abs() <= tol).all())
    y = lib.cache_attention(q[-1:].cuda(), w.cache, w.table, w.lengths, slots=w.slots, window=16)
    assert not bool(y.isnan().any())


def test_attention_strided_queries_and_hints(lib):
    """q as a view into a fused projection; max_len below and above the truth."""
    w = World(lib, [700, 260], 2, 64, 32, "fp16", seed=12)
    fused = torch.full((2, 8, 128), math.nan, dtype=torch.float16)
    q = torch.randn((2, 4, 64), generator=gen(3)).half()
    fused[:, ::2, 64:] = q
    view = fused.cuda()[:, ::2, 64:]
    want = None
    for max_len in (None, 700, 100, 0, 5000):
        y = lib.cache_attention(view, w.cache, w.table, w.lengths, slots=w.slots, max_len=max_len)
        for b, (k, v, s) in enumerate(w.stored()):
            o, tol = O.attention(q[b:b + 1], k, v, 64 ** -0.5, page_scale=s)
            assert bool(((y[b:b + 1].cpu().double() - o).abs() <= tol).all()), max_len


def test_attention_rows_past_max_q_are_not_written(lib):
    """max_q below a sequence's rows: the first rows are right, the others untouched;
    a window past any position is none."""
    w = World(lib, [90, 33], 1, 64, 16, "fp16", seed=21)
    q = torch.randn((12, 2, 64), generator=gen(5)).half().cuda()
    args = (q, w.cache, w.table, w.lengths)
    whole = lib.cache_attention(*args, cu=w.cu([7, 5]), slots=w.slots, window=2 ** 31 - 1)
    out = torch.full_like(q, 7.0)
    lib.cache_attention(*args, cu=w.cu([7, 5]), slots=w.slots, max_q=6, out=out)
    same(out[:6], whole[:6])
    same(out[7:], whole[7:])
    assert bool((out[6] == 7.0).all())


def test_attention_is_deterministic_on_any_stream(lib):
    w = World(lib, [3000, 1, 500], 2, 128, 64, "fp16", seed=13)
    q = torch.randn((3, 4, 128), generator=gen(4)).half().cuda()
    a = lib.cache_attention(q, w.cache, w.table, w.lengths, slots=w.slots)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = lib.cache_attention(q, w.cache, w.table, w.lengths, slots=w.slots)
    s.synchronize()
    same(a, b)


def test_cache_past_32_bit_offsets(lib):
    """Pages behind the 2^31st code, and past 2^32: written, read back and attended."""
    H, D, P = 8, 128, 128
    n = (1 << 32) // (H * D * P) + 8          # 4.3 GB of codes for keys and as much for values
    say("cache with", n, "pages")
    cache = lib.new_cache(n, 1, H, D, P, torch.float16, "cuda:0")
    table = torch.tensor([[n - 1, n // 2 + 3, n - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    g = gen(14)
    k, v = (torch.randn((300, H, D), generator=g).half() for _ in range(2))
    lib.cache_write(cache, k.cuda(), v.cuda(), table, lens,
                    cu=torch.tensor([0, 300], dtype=torch.int32, device="cuda"))
    st = O.Store(P)
    kk, (vv, pages) = st.sequence(k)[0], st.sequence(v)
    rk, rv = lib.cache_read(cache, table, lens,
                            torch.zeros(2, dtype=torch.int32, device="cuda"), 300)
    same(rk, kk.half())
    same(rv, vv.half())
    s = torch.ones((300, H))
    for i, per in enumerate(pages):
        for h, (_, sc) in enumerate(per):
            s[i * P:(i + 1) * P, h] = sc
    q = torch.randn((1, H, D), generator=g).half()
    y = lib.cache_attention(q.cuda(), cache, table, lens)
    o, tol = O.attention(q, kk, vv, D ** -0.5, page_scale=s)
    assert bool(((y.cpu().double() - o).abs() <= tol).all())


def test_decode_steps_in_a_graph(lib):
    """Append, attend and project in a captured graph, replayed with eager work between:
    every replay equals the eager result."""
    B, H, G, D, P, N = 3, 2, 2, 64, 16, 128
    w = World(lib, [40, 17, 32], H, D, P, "fp16", seed=15)
    g = gen(16)
    q = torch.randn((B, H * G, D), generator=g).half().cuda()
    k = torch.randn((B, H, D), generator=g).half().cuda()
    x = torch.randn((B, H * G * D), generator=g).half().cuda()
    Wq = torch.randint(-127, 128, (N, H * G * D), generator=g, dtype=torch.int8).cuda()
    sw = torch.rand(N, generator=g).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens.copy_(w.lengths)

    def step():
        lib.cache_write(w.cache, k, k, w.table, lens, slots=w.slots)
        o = lib.cache_attention(q, w.cache, w.table, lens, slots=w.slots, max_len=4096)
        a, s, h = lib.rmsnorm_quant(o.view(B, -1), residual=x)
        return o, lib.linear_codes(a, s, Wq, sw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, yg = step()
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=g).half())
        k.copy_(torch.randn(k.shape, generator=g).half())
        o, y = step()
        torch.cuda.synchronize()
        og.fill_(math.nan)
        yg.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        same(og, o)
        same(yg, y)
