"""Rotary positions and drafts on the GPU where a call's inputs are unusual: what stays as it
is beside infinities and NaNs."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_positions_gpu import (blank_cache, cu_of, freqs_of, gen, ints, lib, parts_of,  # noqa: E402, F401
                                positions_of, say, within)
from oracle import positions_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def bits(x):
    """The bits of a 16-bit tensor, one pattern for every NaN."""
    x = x.cpu().contiguous()
    return torch.where(x.isnan(), torch.tensor(0x7fff, dtype=torch.int16), x.view(torch.int16))


def same_bits(a, b, what=""):
    eq = bits(a) == bits(b)
    assert bool(eq.all()), f"{what}: {int((~eq).sum())} of {eq.numel()} differ"


# D, pairs, interleaved: aligned halves, pairs, halves through LDS; a part that ends at a
# lane's first element, inside a lane, at its last but one; nothing turned
PARTS = [(64, 16, False), (64, 8, True), (64, 11, True), (80, 10, False), (80, 10, True), (128, 1, False),
         (128, 1, True), (96, 36, False), (96, 47, False), (256, 100, False), (256, 100, True), (64, 0, True),
         (64, 0, False)]


def odd_heads(T, H, D, pairs, dt, g):
    """Heads whose elements past the turned ones are any: infinities, NaNs and zeros of both
    signs beside finite ones, in every place of some head."""
    x = torch.randn((T, H, D), generator=g).to(dt)
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0, 0.0])
    at = torch.randint(0, 9, (T, H, D), generator=g)
    at[..., :2 * pairs] = 9
    for i, v in enumerate(odd):
        x[at == i] = float(v)
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,pairs,inter", PARTS)
def test_what_does_not_turn_stays(lib, D, pairs, inter, dtype):  # noqa: F811
    """Elements past the turned ones come out bit for bit, whatever they and their neighbours
    are, and change nothing among the turned ones: forward and backward."""
    say("what does not turn", D, pairs, inter, dtype)
    dt, g = TYPES[dtype], gen(D + pairs)
    T, H = 40, 3
    x = odd_heads(T, H, D, pairs, dt, g)
    clean = x.clone()
    clean[..., 2 * pairs:] = 1
    f, pos = freqs_of(pairs), torch.randint(0, 1 << 18, (T,), generator=g).to(torch.int32)
    rot = lib.Rotary(f.cuda(), interleaved=inter, factor=1.25)
    for y, (want, tol) in (
            (lib.rotate_heads(x.cuda(), pos.cuda(), rot), O.rotate(clean, pos, f, inter, 1.25)),
            (lib.rotate_heads_backward(x.cuda(), pos.cuda(), rot)[0],
             O.rotate_grad(clean, None, pos, f, inter, 1.25)[0])):
        same_bits(y[..., 2 * pairs:], x[..., 2 * pairs:], "what does not turn")
        n = 2 * pairs
        within(y[..., :n], want[..., :n], tol[..., :n], "what turns")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,pairs,inter", PARTS)
def test_what_does_not_turn_reaches_the_cache(lib, D, pairs, inter, dtype):  # noqa: F811
    """cache_append: queries, and keys in the incomplete page, the same."""
    say("what does not turn, appended", D, pairs, inter, dtype)
    dt, g = TYPES[dtype], gen(D + pairs + 1)
    P, H, n = 64, 2, 37
    c = blank_cache(lib, 1, 1, H, D, P, dt)
    q, k = odd_heads(n, 3, D, pairs, dt, g), odd_heads(n, H, D, pairs, dt, g)
    v = torch.randn((n, H, D), generator=g).to(dt)
    rot = lib.Rotary(freqs_of(pairs).cuda(), interleaved=inter)
    got = lib.cache_append(c, k.cuda(), v.cuda(), ints([[0]]), ints([n]), q=q.cuda(), rotary=rot, cu=ints([0, n]))
    same_bits(got[..., 2 * pairs:], q[..., 2 * pairs:], "queries")
    same_bits(c.k_tail[0].transpose(0, 1)[:n, :, 2 * pairs:], k[..., 2 * pairs:], "keys")


def test_frequencies_changed_before_the_backward_pass(lib):  # noqa: F811
    """Frequencies written over between the passes would give another function's gradient:
    autograd says so, as for any tensor that a backward pass needs."""
    from mixed_precision_quantized_int8_amd.module import RotateHeads

    m = RotateHeads(64, lib.rotary(64))
    q = torch.randn((5, 2, 64), generator=gen(1)).half().cuda().requires_grad_()
    pos = ints(list(range(5)))
    out = m(q, pos)
    m.rotary.freqs.mul_(0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    m(q, pos).sum().backward()                    # (with the new ones from here on)
    want, _, dw, _ = lib.rotate_heads_backward(torch.ones_like(q), pos, m.rotary, q=q.detach(),
                                               q_weight=m.q_weight.detach())
    same_bits(q.grad, want)
    same_bits(m.q_weight.grad, dw)
    with torch.autograd.graph.save_on_cpu():      # what was saved is what counts
        out = m(q, pos)
    m.rotary.freqs.mul_(0.5)
    same_bits(torch.autograd.grad(out.sum(), q)[0], want)
    plain = RotateHeads(64, None)                 # no rotation: nothing to change
    torch.autograd.grad(plain(q, pos).sum(), q)


@pytest.mark.parametrize("P,D,pairs,inter", [(16, 64, 32, False), (64, 128, 64, True), (32, 80, 10, False),
                                             (128, 256, 128, False)])
def test_many_queries_of_short_sequences(lib, P, D, pairs, inter):  # noqa: F811
    """Calls of thousands of rows, none of whose sequences is long: bit for bit rotate_heads and
    cache_write, rows behind the sequences left as they are, whatever bound max_new is."""
    say("many queries", P, D, pairs, inter)
    H, G, dt, g = 1, 3, torch.bfloat16, gen(P + D)
    new = [0, 1, 2, 3, 4, 5, 7, 130] + torch.randint(1, 60, (90,), generator=g).tolist()
    lens = [n + (i % 3) * 9 for i, n in enumerate(new)]
    B, T, per = len(new), sum(new), -(-max(lens) // P)
    assert T > 2048
    rot = lib.Rotary(freqs_of(pairs).cuda(), interleaved=inter)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(dt).cuda()
    q, k, v = torch.randn((T, H * (G + 2), D), generator=g).to(dt).cuda().split([H * G, H, H], dim=1)
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    length, cu, pos = ints(lens), cu_of(new), positions_of(lens, new).cuda()
    a = blank_cache(lib, B * per, B, H, D, P, dt)
    q1, k1 = lib.rotate_heads(q, pos, rot, k=k, q_weight=w, k_weight=w)
    lib.cache_write(a, k1, v, table, length, cu=cu, max_new=130)
    for most in (130, None):
        b = blank_cache(lib, B * per, B, H, D, P, dt)
        out = torch.full((T + 3, H * G, D), 9.0, dtype=dt, device="cuda")
        lib.cache_append(b, k, v, table, length, q=q, rotary=rot, q_weight=w, k_weight=w, cu=cu, max_new=most,
                         q_out=out[:T])
        same_bits(out[:T], q1, "queries")
        assert bool((out[T:] == 9).all())
        for x, y in zip(parts_of(a), parts_of(b)):
            assert torch.equal(x, y)
