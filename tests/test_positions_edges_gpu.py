"""Rotary positions and drafts on the GPU where a call is unusual: what stays as it is beside
infinities and NaNs, frequencies that change, thousands of short sequences, and what is not
finite, hidden or past the bound in trees whose keys are shared out."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_positions_gpu import (blank_cache, check_tree, cu_of, filled_cache, freqs_of, gen,  # noqa: E402, F401
                                ints, lib, parts_of, positions_of, random_tree, say, within)
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


# ---- trees whose keys are shared out to workgroups by their number ------------------

# lens, drafts, H, G, D, P: several segments a workgroup and several workgroups a tile; a
# sequence without keys, one without drafts, two words of mask, tiles whose last is not full
SHARES = [([2500, 0, 700], [70, 33, 64], 2, 4, 128, 16), ([2100, 60, 2300, 5], [66, 40, 0, 64], 3, 8, 64, 64)]


def share_case(lib, case, dt, g):  # noqa: F811
    """(cache, table, slots, per-sequence keys and values, q, k, v, a call) of a batch that is shared."""
    lens, sizes, H, G, D, P = case
    cache, table, slots, kv = filled_cache(lib, lens, H, D, P, dt, g, poison=True)
    q, k, v = torch.randn((sum(sizes), H * (G + 2), D), generator=g).to(dt).cuda().split([H * G, H, H], dim=1)
    most = max(sizes)
    # two places a workgroup for 256 rows' sums and outputs, 192 words before them: the way taken
    assert lib.tree_workspace_bytes(cache, len(lens), H * G, most, max(lens)) == \
        4 * (192 + 2 * (256 // H) * H * 256 * (D + 2))

    def call(masks, k=k, v=v, max_q=most, **kw):
        return lib.tree_attention(q, k, v, cache, table, ints(lens), masks, cu=cu_of(sizes), slots=slots,
                                  max_q=max_q, max_len=max(lens), scale=0.11, **kw)

    return cache, table, slots, kv, q, k, v, call


def tree_masks(sizes, lens, g):
    seen = [O.tree_plan(random_tree(m, g, root=m % 2 == 0), n)[1] for n, m in zip(lens, sizes)]
    return seen, torch.cat([O.words(s, 2) for s in seen if s]).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", SHARES, ids=["three", "four"])
def test_shared_trees_with_non_finite_drafts(lib, case, dtype):  # noqa: F811
    """Infinities and NaNs in a draft's key or value show in the drafts that see it, and in no
    other row of any sequence."""
    lens, sizes, H, G, D, P = case
    say("shared trees, non-finite drafts", case, dtype)
    dt, g = TYPES[dtype], gen(sum(lens))
    cache, table, slots, kv, q, k, v, call = share_case(lib, case, dt, g)
    seen, masks = tree_masks(sizes, lens, g)
    clean = call(masks)
    check_tree(lib, cache, table, slots, kv, lens, None, q, k, v, P, dt, 0.11, 0, None, clean, [0] * q.shape[0], seen)
    first = cu_of(sizes).tolist()
    for bad in (math.nan, math.inf, -math.inf):
        for b, j in ((0, 0), (0, sizes[0] - 1), (1, 2), (len(sizes) - 1, 63)):
            for into in "vk":
                k2, v2 = k.clone(), v.clone()
                (v2 if into == "v" else k2)[first[b] + j, H - 1, 5] = bad
                got = call(masks, k2, v2)
                sees = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
                sees[first[b]:first[b + 1]] = torch.tensor([j in s for s in seen[b]], device="cuda")
                hit = torch.zeros_like(got, dtype=torch.bool)
                if into == "v":
                    hit[:, (H - 1) * G:, 5] = sees[:, None]
                    assert not bool(got[hit].isfinite().any())
                else:      # an infinite score is NaN or hides the key: only rows that see it
                    hit[:, (H - 1) * G:] = sees[:, None, None]
                    if bad != bad:
                        assert bool(got[hit].isnan().all())
                what = f"{bad} in {into} of draft {j} of sequence {b}"
                if into == "v":
                    same_bits(torch.where(hit, 0, got), torch.where(hit, 0, clean), what)
                    continue
                # A wave's rows move their maximum together, when one of them passes it: another
                # key moves where a row's weights are rounded, if a row of its wave sees it (a
                # finite one does so too).  Those rows stay within the oracle's tolerance, which
                # holds for any maximum; other heads and sequences keep their bits.
                near = torch.zeros_like(hit)
                near[first[b]:first[b + 1], (H - 1) * G:] = True
                same_bits(torch.where(near, 0, got), torch.where(near, 0, clean), what)
                check_tree(lib, cache, table, slots, kv, lens, None, q, k, v, P, dt, 0.11, 0, None,
                           torch.where(hit, clean, got), [0] * q.shape[0], seen)


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_trees_with_a_non_finite_tail(lib, dtype):  # noqa: F811
    """The same in a sequence's incomplete page, which all of its drafts see, with tiles of
    other sequences before and after it in a workgroup."""
    case = SHARES[0]
    lens, sizes, H, G, D, P = case
    say("shared trees, non-finite tail", dtype)
    dt, g = TYPES[dtype], gen(7)
    cache, table, slots, kv, q, k, v, call = share_case(lib, case, dt, g)
    seen, masks = tree_masks(sizes, lens, g)
    clean, first = call(masks), cu_of(sizes).tolist()
    for b in (0, 2):       # 2500 and 700 tokens: 4 and 12 in the incomplete page
        for tail, at in ((cache.v_tail, (int(slots[b]), 1, 5, 3)), (cache.k_tail, (int(slots[b]), 1, 3, 5))):
            for bad in (math.nan, math.inf):
                kept = float(tail[at])
                tail[at] = bad
                got = call(masks)
                tail[at] = kept
                hit = torch.zeros_like(got, dtype=torch.bool)
                rows = slice(first[b], first[b + 1])
                if tail is cache.v_tail:
                    hit[rows, G:, 5] = True
                    assert not bool(got[hit].isfinite().any())
                else:
                    hit[rows, G:] = True
                    if bad != bad:
                        assert bool(got[hit].isnan().all())
                same_bits(torch.where(hit, 0, got), torch.where(hit, 0, clean), f"{bad}, sequence {b}")
    same_bits(call(masks), clean)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", SHARES, ids=["three", "four"])
def test_shared_trees_with_any_mask(lib, case, dtype):  # noqa: F811
    """Masks that are no tree: nothing, everything, bits past the drafts; a sequence without
    keys whose masks are empty gives 0; drafts past max_q are neither seen nor answered, and
    rows behind the last sequence are left as they are."""
    lens, sizes, H, G, D, P = case
    say("shared trees, any mask", case, dtype)
    dt, g = TYPES[dtype], gen(sum(lens) + 1)
    cache, table, slots, kv, q, k, v, call = share_case(lib, case, dt, g)
    seen = [[set(torch.nonzero(torch.rand(m, generator=g) < 0.4)[:, 0].tolist()) for _ in range(m)] for m in sizes]
    for s in seen:
        if s:
            s[0], s[1] = set(), set(range(len(s)))
    empty = lens.index(0) if 0 in lens else None
    if empty is not None:
        seen[empty][3:20] = [set()] * 17
    masks = torch.cat([O.words(s, 2) for s in seen if s])
    first = cu_of(sizes).tolist()
    for b, m in enumerate(sizes):        # drafts that there are not
        if m <= 64:
            masks[first[b]:first[b + 1], 1] = -1
        if 0 < m < 64:
            masks[first[b]:first[b + 1], 0] |= -(1 << m)
    masks = masks.cuda()
    rows = sum(sizes)
    out = torch.full((rows + 4, H * G, D), 9.0, dtype=dt, device="cuda")
    got = call(masks, out=out[:rows])
    check_tree(lib, cache, table, slots, kv, lens, None, q, k, v, P, dt, 0.11, 0, None, got, [0] * rows, seen)
    assert bool((out[rows:] == 9).all())
    if empty is not None:
        assert bool((got[first[empty] + 3:first[empty] + 20] == 0).all())
    # fewer answered
    few = 62
    got = call(masks, max_q=few, out=out[:rows].fill_(9.0))
    for b, m in enumerate(sizes):
        at, n = first[b], min(m, few)
        assert bool((got[at + n:at + m] == 9).all())
        if m:
            cut = [[{i for i in s if i < few} for s in seen[b][:n]]]
            one = slice(at, at + n)
            check_tree(lib, cache, table, slots, kv[b:b + 1], lens[b:b + 1], None, q[one], k[one], v[one], P, dt,
                       0.11, 0, None, got[one], [0] * n, cut)


def test_frequencies_made_in_inference_mode_train(lib):  # noqa: F811
    """Frequencies that carry no version (autograd saves no such tensor) serve in training too."""
    from mixed_precision_quantized_int8_amd.module import RotateHeads

    with torch.inference_mode():
        rot = lib.rotary(64)
    q = torch.randn((5, 2, 64), generator=gen(1)).half().cuda().requires_grad_()
    pos = ints(list(range(5)))
    got, want = (torch.autograd.grad(RotateHeads(64, r)(q, pos).float().square().sum(), q)[0]
                 for r in (rot, lib.rotary(64)))
    same_bits(got, want)
