"""Rotary positions and drafted tokens over the 8-bit cache on the GPU, against the CPU
oracle in float64 with tolerances derived from the arithmetic (oracle/positions_oracle.py
states them), and against each other bit for bit where they must give the same.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from oracle import positions_oracle as O  # noqa: E402
from oracle import serving_oracle as S  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


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


def same(a, b, what=""):
    """Equal bit for bit (NaN with NaN)."""
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    eq = a == b
    if a.is_floating_point():
        eq |= a.isnan() & b.isnan()
    assert bool(eq.all()), f"{what}: {int((~eq).sum())} of {eq.numel()} differ"


def within(got, want, tol, what=""):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: error {float(err.max()):.3g}, {float((err / tol.clamp_min(1e-300)).max()):.3g} of the tolerance"


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ---- norm and rotation --------------------------------------------------------------

# rows, q heads, k heads, D, pairs: every lane count, halves at and off multiples of 8 (the
# way through LDS), part of the head, nothing turned; one head, many, more than one wave holds
HEADS = [(1, 32, 8, 128, 64), (3, 1, 1, 16, 8), (5, 3, 2, 16, 3), (2, 5, 5, 32, 16), (7, 4, 1, 48, 12),
         (4, 15, 5, 80, 10), (4, 15, 5, 80, 40), (3, 6, 2, 96, 24), (9, 7, 7, 112, 56), (2, 33, 11, 64, 32),
         (6, 8, 2, 256, 128), (3, 2, 1, 256, 100), (2, 3, 1, 64, 0), (300, 9, 3, 64, 8), (2, 40, 40, 128, 1)]


def heads_case(T, Hq, Hk, D, dtype, seed):
    g = gen(seed)
    qkv = torch.randn((T, Hq + Hk, D), generator=g).to(dtype)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype) for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    pos[0] = 0
    if T > 2:
        qkv[2] = 0           # a row of zeros
        pos[1] = -5
    return qkv[:, :Hq], qkv[:, Hq:], w, pos


def freqs_of(pairs):
    return torch.tensor([10000.0 ** (-i / max(pairs, 1)) for i in range(pairs)], dtype=torch.float32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,pairs", HEADS)
def test_rotate_heads(lib, T, Hq, Hk, D, pairs, inter, dtype):
    say("rotate_heads", T, Hq, Hk, D, pairs, inter, dtype)
    dt = TYPES[dtype]
    q, k, (qw, kw), pos = heads_case(T, Hq, Hk, D, dt, T * 7 + D + pairs)
    f = freqs_of(pairs)
    qd, kd, pd = torch.cat([q, k], dim=1).cuda().split([Hq, Hk], dim=1) + (pos.cuda(),)
    for wq, wk, factor in ((qw, kw, 1.0), (None, None, 1.25), (qw, None, 1.0)):
        rot = lib.Rotary(f.cuda(), interleaved=inter, factor=factor)
        a, b = lib.rotate_heads(qd, pd, rot, k=kd, q_weight=None if wq is None else wq.cuda(),
                                k_weight=None if wk is None else wk.cuda(), eps=1e-5)
        for got, x, w in ((a, q, wq), (b, k, wk)):
            want, tol = O.rotate(x, pos, f, inter, factor, w, 1e-5)
            within(got, want, tol, f"weight {w is not None}")
    alone = lib.rotate_heads(qd, pd, rot, q_weight=qw.cuda(), eps=1e-5)
    same(alone, a)
    same(lib.rotate_heads(kd, pd, rot), b)
    # into tensors with gaps, and in place
    wide = torch.full((T, Hq + Hk + 1, D + 8), 7.0, dtype=dt, device="cuda")
    x, y = lib.rotate_heads(qd, pd, rot, k=kd, q_weight=qw.cuda(), eps=1e-5, q_out=wide[:, :Hq, :D],
                            k_out=wide[:, Hq:Hq + Hk, :D])
    same(x, a)
    same(y, b)
    assert bool((wide[:, -1] == 7).all()) and bool((wide[:, :, D:] == 7).all())
    heads_first = torch.empty((Hq, T, D), dtype=dt, device="cuda").transpose(0, 1)
    same(lib.rotate_heads(qd, pd, rot, q_weight=qw.cuda(), eps=1e-5, q_out=heads_first), a)
    lib.rotate_heads(qd, pd, rot, k=kd, q_weight=qw.cuda(), eps=1e-5, q_out=qd, k_out=kd)
    same(qd, a)
    same(kd, b)


def test_rotate_heads_without_a_rotation(lib):
    q, k, (qw, kw), pos = heads_case(5, 3, 1, 80, torch.float16, 3)
    a, b = lib.rotate_heads(q.cuda(), pos.cuda(), k=k.cuda(), k_weight=kw.cuda())
    same(a, q)
    within(b, *O.rotate(k, pos, torch.zeros(0), weight=kw))


def test_rotate_heads_far_positions(lib):
    """Angles of positions up to the largest, at the fastest frequency."""
    g = gen(5)
    pos = torch.tensor([0, 1, 1000003, 16777217, (1 << 30) + 1, (1 << 31) - 1, -(1 << 31)], dtype=torch.int64)
    x = torch.randn((7, 2, 64), generator=g).half()
    f = torch.rand(32, generator=g)
    f[0] = 1.0
    got = lib.rotate_heads(x.cuda(), pos.to(torch.int32).cuda(), lib.Rotary(f.cuda()))
    within(got, *O.rotate(x, pos, f))


def test_rotate_heads_quarter_turns(lib):
    """Angles around every multiple of an eighth of a turn."""
    n = 64
    f = torch.tensor([2 * math.pi * i / 64 + d for i in range(n) for d in (0.0, 1e-6, -1e-6)][:96],
                     dtype=torch.float32)
    x = torch.randn((3, 5, 256), generator=gen(6)).half()
    pos = torch.tensor([1, -1, 3], dtype=torch.int32)
    got = lib.rotate_heads(x.cuda(), pos.cuda(), lib.Rotary(f.cuda(), interleaved=True))
    within(got, *O.rotate(x, pos, f, True))


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rotate_heads_at_the_ends_of_the_type(lib, eps):
    """bf16 heads whose squares leave fp32 at either end; zeros among them."""
    x = torch.randn((8, 2, 64), generator=gen(7))
    for i, e in enumerate((-120, -80, -60, 0, 50, 70, 120)):
        x[i] *= 2.0 ** e
    x = x.bfloat16()
    x[7] = 0
    w = (1 + 0.3 * torch.randn(64, generator=gen(8))).bfloat16()
    pos = torch.arange(8, dtype=torch.int32)
    f = freqs_of(32)
    got = lib.rotate_heads(x.cuda(), pos.cuda(), lib.Rotary(f.cuda()), q_weight=w.cuda(), eps=eps)
    want, tol = O.rotate(x, pos, f, weight=w, eps=eps)
    within(got, want, tol)
    assert bool((got[7] == 0).all())
    dy = torch.randn(x.shape, generator=gen(9)).bfloat16()
    dx, _, dw, _ = lib.rotate_heads_backward(dy.cuda(), pos.cuda(), lib.Rotary(f.cuda()), q=x.cuda(),
                                             q_weight=w.cuda(), eps=eps)
    (want, tol), (want_w, tol_w) = O.rotate_grad(dy, x, pos, f, weight=w, eps=eps)
    # gradients of the smallest heads pass bf16's range: infinities there
    big = want.abs() > 2.0 ** 127
    within(torch.where(big.cuda(), 0.0, dx), torch.where(big, 0.0, want), tol)
    within(dw, want_w, tol_w)


def test_rotate_heads_non_finite_heads_stay_apart(lib):
    q, k, (qw, kw), pos = heads_case(4, 6, 2, 80, torch.float16, 9)
    rot = lib.Rotary(freqs_of(10).cuda())
    a, b = lib.rotate_heads(q.cuda(), pos.cuda(), rot, k=k.cuda(), q_weight=qw.cuda(), k_weight=kw.cuda())
    q2, k2 = q.clone(), k.clone()
    q2[1, 3, 7], k2[3, 0, 70] = math.nan, math.inf
    c, d = lib.rotate_heads(q2.cuda(), pos.cuda(), rot, k=k2.cuda(), q_weight=qw.cuda(), k_weight=kw.cuda())
    assert bool(c[1, 3].isnan().all()) and bool(d[3, 0].isnan().any())
    c[1, 3], d[3, 0] = a[1, 3], b[3, 0]
    same(c, a)
    same(d, b)


def test_rotate_heads_empty(lib):
    x = torch.zeros((0, 3, 64), dtype=torch.float16, device="cuda")
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    rot = lib.rotary(64)
    assert lib.rotate_heads(x, pos, rot).shape == (0, 3, 64)
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    dx, dk, dw, dkw = lib.rotate_heads_backward(x, pos, rot, q=x, dk=x, k=x, q_weight=w, k_weight=w)
    assert dx.shape == dk.shape == (0, 3, 64)
    assert bool((dw == 0).all()) and bool((dkw == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,pairs", HEADS)
def test_rotate_heads_backward(lib, T, Hq, Hk, D, pairs, inter, dtype):
    say("rotate_heads_backward", T, Hq, Hk, D, pairs, inter, dtype)
    dt = TYPES[dtype]
    q, k, (qw, kw), pos = heads_case(T, Hq, Hk, D, dt, T * 3 + D + pairs)
    g = gen(T + D)
    dq, dk = torch.randn(q.shape, generator=g).to(dt), torch.randn(k.shape, generator=g).to(dt)
    f = freqs_of(pairs)
    dev = [t.cuda() for t in (dq, dk, pos)]
    for wq, wk in ((qw, kw), (None, None), (None, kw)):
        rot = lib.Rotary(f.cuda(), interleaved=inter, factor=1.25)
        out = lib.rotate_heads_backward(dev[0], dev[2], rot, q=q.cuda() if wq is not None else None, dk=dev[1],
                                        k=k.cuda() if wk is not None else None,
                                        q_weight=None if wq is None else wq.cuda(),
                                        k_weight=None if wk is None else wk.cuda(), eps=1e-5)
        for i, (dy, x, w) in enumerate(((dq, q, wq), (dk, k, wk))):
            (want, tol), dw = O.rotate_grad(dy, x, pos, f, inter, 1.25, w, 1e-5)
            within(out[i], want, tol, f"dx {i}")
            if w is None:
                assert out[2 + i] is None
            else:
                within(out[2 + i], *dw, f"dweight {i}")
    # in place, and the same bits again
    again = lib.rotate_heads_backward(dev[0], dev[2], rot, dk=dev[1], k=k.cuda(), k_weight=kw.cuda(), eps=1e-5,
                                      dq_out=dev[0], dk_out=dev[1])
    assert again[0].data_ptr() == dev[0].data_ptr() and again[1].data_ptr() == dev[1].data_ptr()
    for a, b in zip(again, out):
        if b is not None:
            same(a, b)


def test_rotate_heads_backward_many_rows(lib):
    """More rows than one pass of the workgroups: the weights' sums go through many."""
    T, D = 5000, 64
    q, k, (qw, kw), pos = heads_case(T, 8, 2, D, torch.float16, 11)
    g = gen(12)
    dq, dk = torch.randn(q.shape, generator=g).half(), torch.randn(k.shape, generator=g).half()
    f = freqs_of(32)
    out = lib.rotate_heads_backward(dq.cuda(), pos.cuda(), lib.Rotary(f.cuda()), q=q.cuda(), dk=dk.cuda(),
                                    k=k.cuda(), q_weight=qw.cuda(), k_weight=kw.cuda())
    for i, (dy, x, w) in enumerate(((dq, q, qw), (dk, k, kw))):
        (want, tol), dw = O.rotate_grad(dy, x, pos, f, weight=w)
        within(out[i], want, tol)
        within(out[2 + i], *dw)


def test_rotate_heads_module(lib):
    """RotateHeads through autograd: the gradients of the oracle, between quantized layers in
    their training mode; two calls before one backward pass."""
    from mixed_precision_quantized_int8_amd.module import Int8Linear, RotateHeads

    torch.manual_seed(0)
    T, H, D = 9, 4, 32
    rot = lib.rotary(D, interleaved=True)
    m = RotateHeads(D, rot)
    with torch.no_grad():
        m.q_weight.mul_(1.5)
    q = torch.randn((T, H, D), device="cuda").half().requires_grad_()
    k = torch.randn((T, 1, D), device="cuda").half().requires_grad_()
    pos = ints(list(range(T)))
    a, b = m(q, pos, k)
    c, d = m(k, pos), m(q, pos, k)[1]
    ga, gb = torch.randn_like(a), torch.randn_like(b)
    torch.autograd.backward([a, b], [ga, gb])
    f = rot.freqs.cpu()
    for x, dy, w in ((q, ga, m.q_weight), (k, gb, m.k_weight)):
        (dx, tol), (dw, tol_w) = O.rotate_grad(dy.cpu(), x.detach().cpu(), pos.cpu(), f, True,
                                               weight=w.detach().cpu())
        within(x.grad, dx, tol)
        within(w.grad, dw, tol_w)
    # directional differences of the oracle's forward pass in 64 bits
    v = torch.randn(q.shape, generator=gen(1), dtype=torch.float64)
    x, w, h = q.detach().cpu().double(), m.q_weight.detach().cpu().double(), 1e-4
    y = [O.turn(O.norm(x + s * h * v, w, 1e-6), pos.cpu(), f, True) for s in (1, -1)]
    slope = float(((y[0] - y[1]) / (2 * h) * ga.cpu().double()).sum())
    dx, tol = O.rotate_grad(ga.cpu(), q.detach().cpu(), pos.cpu(), f, True, weight=m.q_weight.detach().cpu())[0]
    # (h^2 times third derivatives, a few units of each element: 1e-8 * 1e2 * their number)
    assert abs(slope - float((q.grad.cpu().double() * v).sum())) <= float((tol * v.abs()).sum()) + 1e-3
    with pytest.raises(RuntimeError, match="gradient"):
        lib.rotate_heads(q, pos, rot)
    qkv = Int8Linear.from_linear(torch.nn.Linear(64, (H + 2) * D), has_fp16_weights=True)
    rows = torch.randn((T, 64), device="cuda").half()
    z = qkv(rows).view(T, H + 2, D)
    m.zero_grad()
    a, b = m(z[:, :H], pos, z[:, H:H + 1])
    (a.float().square().sum() + b.float().square().sum() + z[:, H + 1:].float().sum()).backward()
    assert all(bool(p.grad.isfinite().all()) and bool((p.grad != 0).any())
               for p in (qkv.weight16, qkv.bias, m.q_weight, m.k_weight))


def test_rotate_heads_module_in_a_graph(lib):
    """A training step's forward and backward pass of RotateHeads, captured and replayed with
    new contents, eager work between: every replay against eager, on another stream too."""
    from mixed_precision_quantized_int8_amd.module import RotateHeads

    g = gen(3)
    T, H, D = 700, 6, 64
    m = RotateHeads(D, lib.rotary(D), dtype=torch.bfloat16)
    q, k = (torch.randn((T, h, D), generator=g).bfloat16().cuda().requires_grad_() for h in (H, 2))
    dy = [torch.randn((T, h, D), generator=g).bfloat16().cuda() for h in (H, 2)]
    pos = torch.randint(0, 1 << 18, (T,), generator=g).to(torch.int32).cuda()

    def step():
        out = m(q, pos, k)
        return list(out) + list(torch.autograd.grad(out, (q, k, m.q_weight, m.k_weight), dy))

    def eager():
        return [t.detach().clone() for t in step()]      # (no graph of these leaves lives on)

    want = eager()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(eager(), want):
            same(a, b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [t.detach() for t in step()]
    for i in range(3):
        with torch.no_grad():
            q.copy_(torch.randn(q.shape, generator=g).bfloat16())
            m.k_weight.copy_((1 + 0.2 * torch.randn(D, generator=g)).bfloat16())
        dy[0].copy_(torch.randn(dy[0].shape, generator=g).bfloat16())
        want = eager()
        torch.cuda.synchronize()
        graph.replay()
        for a, b in zip(held, want):
            same(a, b, f"replay {i}")


# ---- into the cache -----------------------------------------------------------------


def blank_cache(lib, n_pages, n_slots, H, D, P, dt):
    """A cache of known contents, so that what must not change can be seen."""
    c = lib.new_cache(n_pages, n_slots, H, D, page_size=P, dtype=dt)
    for t in (c.k_codes, c.v_codes):
        t.fill_(3)
    for t in (c.k_scale, c.v_scale, c.k_tail, c.v_tail):
        t.fill_(0.5)
    return c


def parts_of(c):
    return [c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail]


def positions_of(lens, new):
    return torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).to(torch.int32)


def cu_of(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return ints(out)


APPEND = [(16, 64, 32, False, 2, 1), (16, 16, 8, True, 3, 1), (16, 16, 3, False, 1, 2), (32, 80, 10, False, 5, 3),
          (32, 80, 40, False, 2, 2), (64, 96, 48, True, 2, 1), (128, 128, 64, False, 2, 4),
          (128, 256, 128, False, 1, 2), (128, 256, 50, False, 2, 1), (64, 128, 16, True, 8, 4),
          (64, 112, 56, False, 3, 1), (16, 32, 0, False, 1, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P,D,pairs,inter,H,G", APPEND)
def test_cache_append(lib, P, D, pairs, inter, H, G, dtype):
    """Prompts, chunks and single tokens: bit for bit rotate_heads and cache_write."""
    say("cache_append", P, D, pairs, inter, H, G, dtype)
    dt, g = TYPES[dtype], gen(P + D + H)
    rot = lib.Rotary(freqs_of(pairs).cuda(), interleaved=inter, factor=1.25)
    qw, kw = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt).cuda() for _ in range(2)]
    B = 3
    steps = [[P + 3, 2 * P, 5], [1, 1, 1], [P - 4, 0, 2 * P + 1], [1, 1, 1], [3 * P, 7, 1]]
    per = 9
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    slots = ints([2, 0, 1])
    a, b = (blank_cache(lib, B * per, B, H, D, P, dt) for _ in range(2))
    lens = [0] * B
    for i, new in enumerate(steps):
        lens = [n + m for n, m in zip(lens, new)]
        T = sum(new)
        qkv = torch.randn((T, H * (G + 2), D), generator=g).to(dt).cuda()
        if i == 2:
            qkv[T // 2, -1, 0], qkv[T // 3, H * G, 1] = math.nan, math.inf
        q, k, v = qkv.split([H * G, H, H], dim=1)
        one = new == [1, 1, 1]
        cu = None if one else cu_of(new)
        length = ints(lens)
        wq, wk = (qw, kw) if i % 2 == 0 else (None, kw)
        q1, k1 = lib.rotate_heads(q, positions_of(lens, new).cuda(), rot, k=k, q_weight=wq, k_weight=wk)
        lib.cache_write(a, k1, v, table, length, cu=cu, slots=slots, max_new=max(new))
        out = torch.full((T + 2, H * G, D), 9.0, dtype=dt, device="cuda")
        q2 = lib.cache_append(b, k, v, table, length, q=q, rotary=rot, q_weight=wq, k_weight=wk, cu=cu,
                              slots=slots, max_new=max(new), q_out=out[:T])
        same(q2, q1, f"q, step {i}")
        assert bool((out[T:] == 9).all())
        for x, y in zip(parts_of(a), parts_of(b)):
            same(y, x, f"cache, step {i}")


def test_cache_append_without_anything_is_cache_write(lib):
    g = gen(2)
    a, b = (blank_cache(lib, 6, 2, 2, 64, 16, torch.float16) for _ in range(2))
    k, v = (torch.randn((50, 2, 64), generator=g).half().cuda() for _ in range(2))
    table, length, cu = ints([[0, 1, 2], [5, 4, 3]]), ints([30, 20]), ints([0, 30, 50])
    lib.cache_write(a, k, v, table, length, cu=cu)
    assert lib.cache_append(b, k, v, table, length, cu=cu) is None
    for x, y in zip(parts_of(a), parts_of(b)):
        same(y, x)


def test_cache_append_past_the_table_and_bad_pages(lib):
    """Tokens past the page table are skipped and count in the positions; pages and slots
    that the cache does not have are left out; a sequence with more rows than tokens keeps its
    last; queries are turned all the same."""
    g = gen(4)
    H, D, P = 2, 64, 16
    rot = lib.rotary(D)
    a, b = (blank_cache(lib, 5, 3, H, D, P, torch.float16) for _ in range(2))
    new, lens = [40, 20, 10], [40, 20, 4]
    qkv = torch.randn((70, 3 * H, D), generator=g).half().cuda()
    q, k, v = qkv.split([H, H, H], dim=1)
    table = ints([[0, 1], [99, 2], [3, -1]])          # sequence 0: 32 of its 40 tokens
    slots, cu, length = ints([0, 1, 7]), cu_of(new), ints(lens)
    q1, k1 = lib.rotate_heads(q, positions_of(lens, new).cuda(), rot, k=k)
    lib.cache_write(a, k1, v, table, length, cu=cu, slots=slots)
    q2 = lib.cache_append(b, k, v, table, length, q=q, rotary=rot, cu=cu, slots=slots)
    same(q2, q1)
    for x, y in zip(parts_of(a), parts_of(b)):
        same(y, x)


@pytest.mark.parametrize("turned", [False, True])
def test_cache_append_picks_rows(lib, turned):
    """index and counts: the named rows only, as if they had been packed."""
    g = gen(5)
    H, D, P = 3, 80, 16
    rot = lib.rotary(20) if turned else None
    kw = (1 + 0.3 * torch.randn(D, generator=g)).half().cuda() if turned else None
    a, b = (blank_cache(lib, 12, 3, H, D, P, torch.float16) for _ in range(2))
    table = torch.arange(12).view(3, 4).to(torch.int32).cuda()
    old = [14, 30, 16]
    k, v = (torch.randn((60, H, D), generator=g).half().cuda() for _ in range(2))
    for c in (a, b):
        lib.cache_append(c, k, v, table, ints(old), rotary=rot, k_weight=kw, cu=cu_of(old))
    k, v = (torch.randn((40, H, D), generator=g).half().cuda() for _ in range(2))
    pick, counts = [[0, 3, 4], [], [39, 25, 26, 30]], ints([3, 0, 4])
    index = torch.full((40,), -1, dtype=torch.int32)
    for b0, rows in zip((0, 10, 20), pick):
        index[b0:b0 + len(rows)] = torch.tensor(rows, dtype=torch.int32)
    length = ints([n + len(p) for n, p in zip(old, pick)])
    rows = torch.tensor(sum(pick, []), device="cuda")
    lib.cache_append(a, k[rows], v[rows], table, length, rotary=rot, k_weight=kw, cu=cu_of([3, 0, 4]))
    lib.cache_append(b, k, v, table, length, rotary=rot, k_weight=kw, cu=ints([0, 10, 20, 40]), counts=counts,
                     index=index.cuda())
    for x, y in zip(parts_of(a), parts_of(b)):
        same(y, x)
    # entries outside k and v are clamped, counts to the rows that a sequence has
    length = length + ints([2, 1, 0])
    index[:2], index[10] = torch.tensor([1000, -7], dtype=torch.int32), 7
    lib.cache_append(a, k[ints([39, 0, 7], torch.int64)], v[ints([39, 0, 7], torch.int64)], table, length,
                     rotary=rot, k_weight=kw, cu=ints([0, 2, 3, 3]))
    lib.cache_append(b, k, v, table, length, rotary=rot, k_weight=kw, cu=ints([0, 2, 11, 40]),
                     counts=ints([50, 1, -3]), index=torch.cat([index[:2], index[10:11], index[3:]]).cuda())
    for x, y in zip(parts_of(a), parts_of(b)):
        same(y, x)


def test_cache_append_counts_and_queries(lib):
    """counts with queries: the first rows of each sequence, the others left as they are."""
    g = gen(6)
    H, G, D, P = 2, 3, 64, 16
    rot, w = lib.rotary(D, interleaved=True), (1 + 0.3 * torch.randn(D, generator=g)).half().cuda()
    a, b = (blank_cache(lib, 9, 3, H, D, P, torch.float16) for _ in range(2))
    table = torch.arange(9).view(3, 3).to(torch.int32).cuda()
    q, k, v = torch.randn((40, H * (G + 2), D), generator=g).half().cuda().split([H * G, H, H], dim=1)
    counts, first = [7, 0, 18], [0, 10, 20]
    lens = [20, 5, 18]
    rows = torch.cat([torch.arange(f, f + n) for f, n in zip(first, counts)]).cuda()
    q1 = lib.cache_append(a, k[rows], v[rows], table, ints(lens), q=q[rows], rotary=rot, q_weight=w, k_weight=w,
                          cu=cu_of(counts))
    out = torch.full((40, H * G, D), 9.0, dtype=torch.float16, device="cuda")
    lib.cache_append(b, k, v, table, ints(lens), q=q, rotary=rot, q_weight=w, k_weight=w,
                     cu=ints([0, 10, 20, 40]), counts=ints(counts), q_out=out)
    same(out[rows], q1)
    left = torch.ones(40, dtype=torch.bool, device="cuda")
    left[rows] = False
    assert bool((out[left] == 9).all())
    for x, y in zip(parts_of(a), parts_of(b)):
        same(y, x)


@pytest.mark.parametrize("n", [64, 65, 300])
def test_tree_attention_of_many_sequences(lib, n):
    """As many sequences as a share's plan holds, and more."""
    g = gen(n)
    H, G, D, P, dt = 1, 8, 64, 32, torch.float16
    lens = [2100] + torch.randint(0, 90, (n - 1,), generator=g).tolist()
    sizes = [40] + torch.randint(0, 6, (n - 1,), generator=g).tolist()
    cache, table, slots, kv = filled_cache(lib, lens, H, D, P, dt, g, poison=True)
    q, k, v = torch.randn((sum(sizes), H * (G + 2), D), generator=g).to(dt).cuda().split([H * G, H, H], dim=1)
    positions, seen = [], []
    for m, size in zip(lens, sizes):
        p, s = O.tree_plan(random_tree(size, g), m)
        positions += p
        seen.append(s)
    masks = torch.cat([O.words(s, 1) for s in seen if s]).cuda()
    got = lib.tree_attention(q, k, v, cache, table, ints(lens), masks, cu=cu_of(sizes), slots=slots,
                             max_q=40, max_len=2100, scale=0.15)
    check_tree(lib, cache, table, slots, kv, lens, None, q, k, v, P, dt, 0.15, 0, None, got, positions, seen)


def test_tree_attention_positions_anywhere(lib):
    """Positions at the ends of 32 bits: no key, or all of them, in a window."""
    g = gen(12)
    H, G, D, P, n, dt = 1, 8, 64, 16, 50, torch.float16
    for m in (2, 30):
        cache, table, slots, kv = filled_cache(lib, [n], H, D, P, dt, g)
        q, k, v = torch.randn((m, H * (G + 2), D), generator=g).to(dt).cuda().split([H * G, H, H], dim=1)
        positions = [2 ** 31 - 1, -2 ** 31] * (m // 2)
        masks = torch.full((m, 1), (1 << m) - 1, dtype=torch.int64, device="cuda")
        got = lib.tree_attention(q, k, v, cache, table, ints([n]), masks, positions=ints(positions), cu=ints([0, m]),
                                 slots=slots, max_q=m, scale=0.2, window=9)
        at = [2 ** 30, -2 ** 29] * (m // 2)           # as the kernels take them
        check_tree(lib, cache, table, slots, kv, [n], None, q, k, v, P, dt, 0.2, 9, None, got, at,
                   [[set(range(m))] * m])


# ---- trees --------------------------------------------------------------------------


def random_tree(n, g, root=True):
    p = []
    for j in range(n):
        lo = max(0, j - 5)
        p.append(-1 if j == 0 else int(torch.randint(lo, j, (1,), generator=g)))
        if not root and j % 7 == 3:
            p[-1] = -1
    return p


@pytest.mark.parametrize("sizes", [[1], [26], [5, 0, 64, 1], [65, 128, 3], [512, 100], [300] * 5])
@pytest.mark.parametrize("first", [False, True])
def test_tree_plan_and_accept(lib, sizes, first):
    g = gen(sum(sizes))
    parents, tokens, choices, tree = [], [], [], []
    for n in sizes:
        p = random_tree(n, g, root=not first)
        if n > 20:
            p[10], p[11] = 11, -9      # no earlier draft: behind the text
        t = torch.randint(0, 3, (n,), generator=g).tolist()
        c = torch.randint(0, 3, (n,), generator=g).tolist()
        tree.append((p, t, c))
        parents += p
        tokens += t
        choices += c
    lens = [10 * i for i in range(len(sizes))]
    starts = torch.randint(0, 3, (len(sizes),), generator=g).tolist()
    rows, words = len(parents), -(-max(sizes) // 64)
    cu = cu_of(sizes)
    pos = torch.full((rows + 1,), -7, dtype=torch.int32, device="cuda")
    positions, masks = lib.tree_plan(ints(parents), ints(lens), cu=cu, max_q=max(sizes), positions=pos[:rows])
    assert masks.shape == (rows, words) and int(pos[rows]) == -7
    path, counts, longer, after = lib.tree_accept(ints(parents), ints(tokens, torch.int64),
                                                  ints(choices, torch.int64), ints(lens), cu=cu,
                                                  first=ints(starts, torch.int64) if first else None,
                                                  max_q=max(sizes))
    at = 0
    for i, (p, t, c) in enumerate(tree):
        want, seen = O.tree_plan(p, lens[i])
        assert positions[at:at + len(p)].tolist() == want
        same(masks[at:at + len(p)], O.words(seen, words))
        got, token = O.tree_accept(p, t, c, starts[i] if first else None)
        assert path[at:at + len(p)].tolist() == [at + j for j in got] + [-1] * (len(p) - len(got))
        assert (int(counts[i]), int(longer[i]), int(after[i])) == (len(got), lens[i] + len(got), token)
        at += len(p)


def test_tree_plan_without_cu_and_a_long_chain(lib):
    positions, masks = lib.tree_plan(ints([-1, -1]), ints([4, 9]))
    assert positions.tolist() == [4, 9] and masks.tolist() == [[1], [1]]
    n = 512
    positions, masks = lib.tree_plan(ints(list(range(-1, n - 1))), ints([100]), cu=ints([0, n]))
    assert positions.tolist() == list(range(100, 100 + n))
    same(masks, O.words([set(range(j + 1)) for j in range(n)], 8))
    path, counts, longer, after = lib.tree_accept(ints(list(range(-1, n - 1))), ints([5] * n, torch.int64),
                                                  ints([5] * n, torch.int64), ints([100]), cu=ints([0, n]))
    assert path.tolist() == list(range(n)) and longer.tolist() == [612] and after.tolist() == [5]


def filled_cache(lib, lens, H, D, P, dt, g, poison=False):
    """(cache, table, slots, per-sequence 16-bit keys and values)."""
    B = len(lens)
    per = max(1, -(-max(lens) // P))
    cache = lib.new_cache(B * per + 1, B, H, D, page_size=P, dtype=dt)
    if poison:      # what no token has written must not show
        cache.k_tail.fill_(math.nan)
        cache.v_tail.fill_(math.inf)
        cache.k_scale.fill_(math.nan)
        cache.v_scale.fill_(math.nan)
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    slots = torch.randperm(B, generator=g).to(torch.int32).cuda()
    kv = [[torch.randn((n, H, D), generator=g).to(dt) for _ in range(2)] for n in lens]
    if sum(lens):
        k, v = (torch.cat([s[i] for s in kv]).cuda() for i in range(2))
        lib.cache_write(cache, k, v, table, ints(lens), cu=cu_of(lens), slots=slots)
    return cache, table, slots, kv


def check_tree(lib, cache, table, slots, kv, lens, trees, q, k, v, P, dt, scale, window, slopes, out, positions,
               masks):
    """Every sequence against the oracle; masks as Python sets per draft."""
    at = 0
    for b, (n, seen) in enumerate(zip(lens, masks)):
        m = len(seen)
        vals, scales = [], []
        for i in range(2):
            x, pages = S.Store(P).sequence(kv[b][i])
            vals.append(torch.cat([x, (k, v)[i][at:at + m].cpu().float()]))
            if i == 1:
                sc = torch.ones((n + m, x.shape[1]), dtype=torch.float64)
                for gg, page in enumerate(pages):
                    sc[gg * P:(gg + 1) * P] = torch.tensor([float(s) for _, s in page], dtype=torch.float64)
                scales = sc
        pos = torch.tensor(positions[at:at + m])
        back = pos[:, None] - torch.cat([torch.arange(n), pos])[None]
        vis = torch.zeros((m, n + m), dtype=torch.bool)
        vis[:, :n] = True
        for j, s in enumerate(seen):
            for i in s:
                vis[j, n + i] = True
        if window:
            vis &= back < window
        want, tol = O.tree_attention(q[at:at + m].cpu(), vals[0], vals[1], scale, vis, back, slopes, scales, dt)
        within(out[at:at + m], want, tol, f"sequence {b}")
        at += m


# lens, drafts, H, G, D, P, window, alibi: both kernels and widths, one draft, more than a tile of
# them, no cached token, pages that end inside a tile, splits whose ranges are empty
TREES = [([100], [26], 8, 4, 128, 16, 0, False), ([37], [1], 2, 1, 64, 16, 0, False),
         ([0, 5, 300], [7, 3, 12], 2, 3, 64, 32, 0, True), ([1000, 20], [70, 40], 2, 2, 80, 64, 0, False),
         ([129, 64, 1], [16, 16, 16], 1, 1, 96, 128, 0, True), ([700, 90], [64, 9], 3, 8, 128, 16, 0, False),
         ([2000], [130], 1, 4, 128, 64, 0, True), ([513], [20], 2, 2, 256, 32, 0, False),
         ([300, 17], [40, 130], 1, 8, 256, 16, 0, True), ([4000, 900], [16, 9], 4, 1, 128, 64, 0, True),
         ([9000], [12], 2, 2, 64, 128, 700, False), ([3000, 10, 2], [30, 70, 5], 2, 4, 128, 32, 100, True),
         ([640], [200], 1, 1, 112, 16, 64, False), ([500, 3], [90, 20], 2, 1, 16, 16, 9, False),
         ([5000], [300], 1, 1, 128, 128, 0, False), ([257] * 5, [2, 0, 1, 33, 8], 2, 2, 64, 32, 3, True),
         ([6000, 5000], [150, 129], 1, 2, 128, 128, 0, True)]
# keys shared out to workgroups by their number: several segments a workgroup, several
# workgroups a tile, tiles without keys or drafts, two tiles of rows, any number of heads
SHARED = [([2500, 130, 0, 700], [70, 33, 5, 64], 2, 4, 128, 16, 0, False),
          ([3000, 64, 2100], [64, 0, 80], 5, 3, 64, 64, 0, True),
          ([2200] + [100, 0, 257, 1] * 6, [40, 3, 20, 64, 0] * 5, 1, 8, 80, 32, 0, False),
          ([9000, 5000], [150, 129], 1, 2, 128, 128, 0, True), ([2300, 2300], [33, 40], 7, 4, 96, 64, 0, False)]
TREES += SHARED


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", TREES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_tree_attention(lib, case, dtype):
    lens, sizes, H, G, D, P, window, alibi = case
    say("tree_attention", *case, dtype)
    dt, g = TYPES[dtype], gen(sum(lens) + sum(sizes) + D)
    cache, table, slots, kv = filled_cache(lib, lens, H, D, P, dt, g, poison=True)
    T = sum(sizes)
    qkv = torch.randn((T, H * (G + 2), D), generator=g).to(dt).cuda()
    q, k, v = qkv.split([H * G, H, H], dim=1)
    positions, seen, words = [], [], -(-max(sizes) // 64)
    for n, m in zip(lens, sizes):
        p, s = O.tree_plan(random_tree(m, g, root=m % 2 == 0), n)
        positions += p
        seen.append(s)
    masks = torch.cat([O.words(s, words) for s in seen]).cuda()
    slopes = torch.tensor([2.0 ** -(1 + 8 * (i + 1) / (H * G)) for i in range(H * G)]) if alibi else None
    out = torch.full((T + 3, H * G, D), 9.0, dtype=dt, device="cuda")
    if case in SHARED:     # two places a workgroup for 256 rows' sums and outputs, 192 words before them
        assert lib.tree_workspace_bytes(cache, len(lens), H * G, max(sizes), max(lens)) == \
            4 * (192 + 2 * (256 // H) * H * 256 * (D + 2))
    got = lib.tree_attention(q, k, v, cache, table, ints(lens), masks, positions=ints(positions), cu=cu_of(sizes),
                             slots=slots, max_q=max(sizes), max_len=max(lens), scale=0.11, window=window,
                             alibi=None if slopes is None else slopes.cuda(), out=out[:T])
    assert bool((out[T:] == 9).all())
    check_tree(lib, cache, table, slots, kv, lens, None, q, k, v, P, dt, 0.11, window, slopes, got, positions, seen)
    if not window and not alibi:      # positions do not matter then
        same(lib.tree_attention(q, k, v, cache, table, ints(lens), masks, cu=cu_of(sizes), slots=slots,
                                max_q=max(sizes), max_len=max(lens), scale=0.11), got)


@pytest.mark.parametrize("G,m", [(1, 9), (8, 30)])
def test_tree_attention_any_mask(lib, G, m):
    """Masks that are no tree: nothing, everything, itself left out, bits past the drafts;
    positions in any order, with a window; drafts past max_q are neither seen nor answered."""
    g = gen(m)
    H, D, P, n, dt = 2, 64, 16, 200, torch.float16
    cache, table, slots, kv = filled_cache(lib, [n], H, D, P, dt, g, poison=True)
    q, k, v = torch.randn((m, H * (G + 2), D), generator=g).to(dt).cuda().split([H * G, H, H], dim=1)
    seen = [set(torch.nonzero(torch.rand(m, generator=g) < 0.4)[:, 0].tolist()) for _ in range(m)]
    seen[0], seen[1] = set(), set(range(m))
    masks = O.words(seen, 2)
    masks[:, 1] = -1                                    # drafts 64 .. 127: there are none
    masks[1, 0] = -1
    positions = torch.randint(150, 260, (m,), generator=g).tolist()
    positions[2] = 900                                  # its window: only the drafts as far behind
    for window in (0, 40):
        got = lib.tree_attention(q, k, v, cache, table, ints([n]), masks.cuda(), positions=ints(positions),
                                 cu=ints([0, m]), slots=slots, max_q=m, scale=0.2, window=window)
        check_tree(lib, cache, table, slots, kv, [n], None, q, k, v, P, dt, 0.2, window, None, got, positions, [seen])
    few = m - 3
    out = torch.full((m, H * G, D), 9.0, dtype=dt, device="cuda")
    got = lib.tree_attention(q, k, v, cache, table, ints([n]), masks.cuda(), cu=ints([0, m]), slots=slots,
                             max_q=few, scale=0.2, out=out)
    assert bool((got[few:] == 9).all())
    check_tree(lib, cache, table, slots, kv, [n], None, q, k, v, P, dt, 0.2, 0, None, got[:few], positions[:few],
               [[{i for i in s if i < few} for s in seen[:few]]])


@pytest.mark.parametrize("G,m", [(1, 16), (8, 40)])
def test_tree_attention_with_nothing_to_see(lib, G, m):
    """No cached token and an empty mask: zeros, in a batch with others; a window that
    leaves nothing too."""
    g = gen(m)
    H, D, P = 2, 64, 16
    cache, table, slots, kv = filled_cache(lib, [0, 50], H, D, P, torch.float16, g, poison=True)
    q, k, v = torch.randn((2 * m, H * (G + 2), D), generator=g).half().cuda().split([H * G, H, H], dim=1)
    masks = torch.zeros((2 * m, 1), dtype=torch.int64, device="cuda")
    cu = ints([0, m, 2 * m])
    got = lib.tree_attention(q, k, v, cache, table, ints([0, 50]), masks, cu=cu, slots=slots, max_q=m)
    assert bool((got[:m] == 0).all()) and bool((got[m:] != 0).any()) and bool(got.isfinite().all())
    got = lib.tree_attention(q, k, v, cache, table, ints([0, 50]), masks, positions=ints([1000] * 2 * m), cu=cu,
                             slots=slots, max_q=m, window=5)
    assert bool((got == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,m", [(1, 12), (8, 40)])
def test_tree_attention_non_finite(lib, G, m, dtype):
    """Infinities and NaNs in a draft's key or value show in the drafts that see it, and in
    no other row."""
    dt, g = TYPES[dtype], gen(m + 1)
    H, D, P, n = 2, 80, 16, 90
    cache, table, slots, kv = filled_cache(lib, [n], H, D, P, dt, g)
    q, k, v = torch.randn((m, H * (G + 2), D), generator=g).to(dt).cuda().split([H * G, H, H], dim=1)
    p, seen = O.tree_plan(random_tree(m, g), n)
    masks = O.words(seen, 1).cuda()

    def run(k, v):
        return lib.tree_attention(q, k, v, cache, table, ints([n]), masks, cu=ints([0, m]), slots=slots, max_q=m)

    clean = run(k, v)
    for bad in (math.nan, math.inf, -math.inf):
        for j in (m - 1, 2):
            for into in "vk":
                k2, v2 = k.clone(), v.clone()
                (v2 if into == "v" else k2)[j, 1, 5] = bad
                got = run(k2, v2)
                sees = torch.tensor([j in s for s in seen], device="cuda")
                hit = torch.zeros_like(got, dtype=torch.bool)
                if into == "v":
                    hit[:, G:, 5] = sees[:, None]
                    assert not bool(got[hit].isfinite().any())
                    assert bool(got[hit].isnan().all()) or bool((got[hit] == bad).all())
                else:      # an infinite score is NaN or hides the key: only rows that see it
                    hit[:, G:] = sees[:, None, None]
                same(torch.where(hit, 0, got), torch.where(hit, 0, clean), f"{bad} in {into} of draft {j}")


def test_tree_attention_of_a_chain_is_cache_attention(lib):
    """A chain's attention and cache_attention after its tokens were appended: the same
    function, up to the rounding of the tokens that a page codes (none here: they stay in
    the tail)."""
    g = gen(3)
    H, G, D, P, n, m = 2, 4, 128, 64, 130, 20
    cache, table, slots, kv = filled_cache(lib, [n], H, D, P, torch.float16, g)
    q, k, v = torch.randn((m, H * (G + 2), D), generator=g).half().cuda().split([H * G, H, H], dim=1)
    positions, masks = lib.tree_plan(ints(list(range(-1, m - 1))), ints([n]), cu=ints([0, m]))
    a = lib.tree_attention(q, k, v, cache, table, ints([n]), masks, positions=positions, cu=ints([0, m]),
                           slots=slots)
    lib.cache_write(cache, k, v, table, ints([n + m]), cu=ints([0, m]), slots=slots)
    b = lib.cache_attention(q, cache, table, ints([n + m]), cu=ints([0, m]), slots=slots)
    vals = [torch.cat([S.Store(P).sequence(x)[0], y.cpu().float()]) for x, y in zip(kv[0], (k, v))]
    vis = torch.arange(n, n + m)[:, None] >= torch.arange(n + m)[None]
    want, tol = O.tree_attention(q.cpu(), vals[0], vals[1], D ** -0.5, vis)
    within(a, want, tol)
    within(b, want, tol)


def test_calls_on_another_stream_and_in_a_graph(lib):
    """The calls together, as a serving step makes them: on a stream of their own, and
    captured, replayed with new contents between eager work; every replay against eager."""
    g = gen(8)
    H, G, D, P, m, n = 2, 4, 64, 16, 14, 700
    cache, table, slots, kv = filled_cache(lib, [n, 45], H, D, P, torch.float16, g)
    save = [t.clone() for t in parts_of(cache)]
    rot, w = lib.rotary(D), (1 + 0.3 * torch.randn(D, generator=g)).half().cuda()
    qkv = torch.randn((2 * m, H * (G + 2), D), generator=g).half().cuda()
    parents = ints(random_tree(m, g) + random_tree(m, g))
    tokens, choices = (torch.randint(0, 2, (2 * m,), generator=g).cuda() for _ in range(2))
    lens, cu = ints([n, 45]), ints([0, m, 2 * m])
    table = torch.cat([table, table.flip(0)], dim=1).contiguous()[:, :table.shape[1]].contiguous()

    def step():
        q, k, v = qkv.split([H * G, H, H], dim=1)
        positions, masks = lib.tree_plan(parents, lens, cu=cu, max_q=m)
        q, k = lib.rotate_heads(q, positions, rot, k=k, q_weight=w, k_weight=w)
        o = lib.tree_attention(q, k, v, cache, table, lens, masks, positions=positions, cu=cu, slots=slots,
                               max_q=m, max_len=n, window=300)
        path, counts, longer, after = lib.tree_accept(parents, tokens, choices, lens, cu=cu, max_q=m)
        lib.cache_append(cache, k, v, table, longer, cu=cu, slots=slots, counts=counts, index=path, max_new=m)
        dq, dk, dw, _ = lib.rotate_heads_backward(q, positions, rot, q=q, dk=k, q_weight=w)
        return positions, masks, q, k, o, counts, longer, after, dq, dk, dw

    def restore():
        for t, s in zip(parts_of(cache), save):
            t.copy_(s)

    def eager():
        restore()
        out = [t.clone() for t in step()]
        return out + [t.clone() for t in parts_of(cache)]

    want = eager()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        other = eager()
    torch.cuda.current_stream().wait_stream(stream)
    for a, b in zip(other, want):
        same(a, b)
    graph = torch.cuda.CUDAGraph()
    restore()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        qkv.copy_(torch.randn(qkv.shape, generator=g).half())
        tokens.copy_(torch.randint(0, 2, (2 * m,), generator=g))
        want = eager()
        torch.cuda.synchronize()
        restore()
        graph.replay()
        for a, b in zip([*held, *parts_of(cache)], want):
            same(a, b, f"replay {i}")


def test_wrappers_refuse_on_the_gpu(lib):
    x = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    rot = lib.rotary(64)
    for bad, err in ((dict(q=x[:, :, :62]), lib.Int8LinError), (dict(q=x[0]), ValueError),
                     (dict(positions=pos[:3]), ValueError), (dict(positions=pos.long()), TypeError),
                     (dict(k=x.bfloat16()), TypeError), (dict(k=x[:3]), ValueError),
                     (dict(k_weight=x[0, 0]), ValueError), (dict(q_weight=x[0, 0].float()), TypeError),
                     (dict(q_weight=x[0, 0, :32]), ValueError), (dict(q_out=x[:2]), ValueError),
                     (dict(rotary=7), TypeError), (dict(rotary=lib.rotary(128)), lib.Int8LinError),
                     (dict(eps=-1.0), lib.Int8LinError), (dict(q=x.transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            lib.rotate_heads(**{**dict(q=x, positions=pos, rotary=rot), **bad})
    w = x[0, 0].contiguous()
    for bad in (dict(q_weight=w), dict(k_weight=w), dict(dk=x, k_weight=w)):
        with pytest.raises(ValueError):
            lib.rotate_heads_backward(x, pos, rot, **bad)
    with pytest.raises(lib.Int8LinError, match="WORKSPACE"):
        lib.rotate_heads_backward(x, pos, rot, q=x, q_weight=w,
                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(AttributeError):
        rot.factor = 2.0
    cache = lib.new_cache(4, 4, 2, 64, page_size=16)
    table, lens = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), pos + 1
    for bad, err in ((dict(k=x[:3]), ValueError), (dict(index=pos, q=x), ValueError),
                     (dict(index=pos[:3]), ValueError), (dict(counts=pos[:2]), ValueError),
                     (dict(q_weight=w), ValueError), (dict(v=x.bfloat16()), TypeError)):
        with pytest.raises(err):
            lib.cache_append(**{**dict(cache=cache, k=x, v=x, page_table=table, lengths=lens, rotary=rot), **bad})
    masks = torch.zeros((4, 1), dtype=torch.int64, device="cuda")
    for bad, err in ((dict(masks=masks[:2]), ValueError), (dict(masks=masks.int()), TypeError),
                     (dict(window=4), lib.Int8LinError), (dict(k=x[:, :1]), ValueError),
                     (dict(max_q=65), lib.Int8LinError), (dict(positions=pos[:1]), ValueError),
                     (dict(q=x[:, :1]), lib.Int8LinError)):
        with pytest.raises(err):
            lib.tree_attention(**{**dict(q=x, k=x, v=x, cache=cache, page_table=table, lengths=lens, masks=masks),
                                  **bad})
    with pytest.raises(ValueError):
        lib.tree_plan(pos, lens[:3])
    with pytest.raises(TypeError):
        lib.tree_accept(pos, pos, pos, lens)


def test_gradients_that_start_anywhere(lib):
    """A gradient that autograd hands on as a view (of a concatenation's, say) may start at any
    element, or have strides of 0."""
    from mixed_precision_quantized_int8_amd.module import RotateHeads

    g = gen(5)
    T, H, D = 7, 3, 64
    m = RotateHeads(D, lib.rotary(D))
    q, k = (torch.randn((T, h, D), generator=g).half().cuda().requires_grad_() for h in (H, 1))
    pos, odd = ints(list(range(T))), torch.zeros(3, dtype=torch.float16, device="cuda")
    w = torch.randn(3 + T * (H + 1) * D, generator=g).half().cuda()
    a, b = m(q, pos, k)
    torch.cat([odd, a.flatten(), b.flatten()]).backward(w)
    got = [q.grad, k.grad, m.q_weight.grad, m.k_weight.grad]
    n = T * H * D
    want = lib.rotate_heads_backward(w[3:3 + n].view(T, H, D).clone(), pos, m.rotary, q=q.detach(),
                                     dk=w[3 + n:].view(T, 1, D).clone(), k=k.detach(),
                                     q_weight=m.q_weight.detach(), k_weight=m.k_weight.detach())
    for x, y in zip(got, want):
        same(x, y)
    dq = torch.autograd.grad(m(q, pos).sum(), q)[0]
    same(dq, lib.rotate_heads_backward(torch.ones_like(q), pos, m.rotary, q=q.detach(),
                                       q_weight=m.q_weight.detach())[0])
