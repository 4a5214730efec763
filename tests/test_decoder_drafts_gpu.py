"""The 8-bit decoder layer with rotary positions and head norms on the GPU: prompts,
single tokens and trees of drafted tokens over one paged cache, against the same layer
in float64 on the unquantized weights."""
import math

import pytest

torch = pytest.importorskip("torch")

from oracle import positions_oracle as O  # noqa: E402
from test_decoder_gpu import D, HEADS, HIDDEN, KV, parts  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(i8l):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return i8l


def reference(p, x, freqs, interleaved, q_norm, k_norm):
    """y and r' [rows] in float64 of one whole sequence's rows."""
    norm1, qkv, out, norm2, up, down = p
    f = lambda lin, v: v @ lin.weight.detach().double().T + (0 if lin.bias is None else  # noqa: E731
                                                            lin.bias.detach().double())
    norm = lambda v, w: v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5) * w.double()  # noqa: E731
    r = x.double()
    n = r.shape[0]
    z = f(qkv, norm(r, norm1)).view(n, HEADS + 2 * KV, D)
    pos = torch.arange(n)
    q, k = (O.turn(O.norm(h, None if w is None else w.double(), 1e-6), pos, freqs, interleaved)
            for h, w in ((z[:, :HEADS], q_norm), (z[:, HEADS:HEADS + KV], k_norm)))
    hide = pos[:, None] < pos[None]
    o = torch.empty((n, HEADS, D), dtype=torch.float64)
    for h in range(HEADS):
        kv = h // (HEADS // KV)
        s = q[:, h] @ k[:, kv].T * D ** -0.5
        o[:, h] = torch.softmax(s.masked_fill(hide, -math.inf), 1) @ z[:, HEADS + KV + kv]
    r = r + f(out, o.view(n, HEADS * D))
    return f(down, torch.nn.functional.gelu(f(up, norm(r, norm2)))), r


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def close(got, want, what):
    # Each 8-bit operand is within half a step of absmax / 127, about 1 % of a normal row's
    # rms (absmax ~ 3.3 rms: 0.5 / 127 * 3.3 = 1.3 %, uniform: / sqrt 3).  A product of two
    # such operands errs by 1.1 % of its rms; four of them in a row, and the cache's two,
    # stay below 3 % together (errors add in squares; norm and rotation keep lengths).
    rel = float((got.cpu().double() - want).norm() / want.norm())
    assert rel < 0.03, f"{what}: {rel:.4f}"


@pytest.mark.parametrize("codes,interleaved,normed", [(False, False, True), (True, True, False),
                                                      (True, False, True)])
def test_prompts_tokens_and_drafts(lib, codes, interleaved, normed):
    from mixed_precision_quantized_int8_amd.decoder import Int8DecoderLayer

    print("decoder layer with drafts, codes", codes, "interleaved", interleaved, "norms", normed, flush=True)
    p, g = parts(6), torch.Generator().manual_seed(7)
    rot = lib.rotary(D // 2 if interleaved else D, interleaved=interleaved)
    freqs = rot.freqs.cpu()
    w = [1 + 0.2 * torch.randn(D, generator=g) for _ in range(2)] if normed else [None, None]
    layer = Int8DecoderLayer(*p, heads=HEADS, kv_heads=KV, codes=codes, rotary=rot, q_norm=w[0], k_norm=w[1])
    B, P, per = 3, 16, 8
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    caches = [lib.new_cache(B * per, B, KV, D, page_size=P) for _ in range(2)]
    for c in caches:
        for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale, c.k_tail, c.v_tail):
            t.zero_()
    cache, other = caches
    text = [torch.randn((n, HIDDEN), generator=g).half() for n in (60, 33, 16)]

    def rows(lo, hi):
        return torch.cat([s[a:b] for s, a, b in zip(text, lo, hi)]).cuda()

    def cu(n):
        return ints([0, n[0], n[0] + n[1], sum(n)])

    def check(got, lo, hi, name):
        at = 0
        for b in range(B):
            y, r = reference(p, text[b], freqs, interleaved, *w)
            m = hi[b] - lo[b]
            for got_x, want in zip(got, (y, r)):
                close(got_x[at:at + m], want[lo[b]:hi[b]], f"{name}, sequence {b}")
            at += m

    lens = [40, 20, 3]
    for c in caches:
        got = layer(rows([0] * 3, lens), None, c, table, ints(lens), cu=cu(lens), max_q=40, max_len=64)
    check(got, [0] * 3, lens, "prompt")
    for _ in range(2):                                       # single tokens
        nxt = [n + 1 for n in lens]
        for c in caches:
            got = layer(rows(lens, nxt), None, c, table, ints(nxt), max_len=64)
        check(got, lens, nxt, "token")
        lens = nxt

    # trees: the text's next rows are one path of each, the other drafts lead elsewhere
    parents = [[-1, 0, 0, 2, 1, 3, 5], [-1, 0, 1, 2], [-1, 0, 0, 0]]
    right = [[0, 2, 3, 5], [0, 1], [0, 3]]                   # drafts that are the text
    held = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_tail, cache.v_tail)]
    drafts, tokens, choices = [], [], []
    for b in range(B):
        x = torch.randn((len(parents[b]), HIDDEN), generator=g).half()
        tok, cho = list(range(100, 100 + len(x))), [0] * len(x)
        for i, j in enumerate(right[b]):
            x[j] = text[b][lens[b] + i]
            if i + 1 < len(right[b]):
                cho[j] = tok[right[b][i + 1]]
        drafts.append(x)
        tokens += tok
        choices += cho
    n = [len(x) for x in drafts]
    positions, masks = lib.tree_plan(ints(sum(parents, [])), ints(lens), cu=cu(n), max_q=max(n))
    y, r, kv = layer.draft(torch.cat(drafts).cuda(), None, cache, table, ints(lens), positions, masks, cu=cu(n),
                           max_q=max(n), max_len=64)
    for a, t in zip(held, (cache.k_codes, cache.v_codes, cache.k_tail, cache.v_tail)):
        assert torch.equal(a, t)                             # drafts are no part of the cache
    at = 0
    for b in range(B):
        for j in range(n[b]):
            line, i = [], j
            while i >= 0:
                line.append(drafts[b][i])
                i = parents[b][i]
            want = reference(p, torch.cat([text[b][:lens[b]], torch.stack(line[::-1])]), freqs, interleaved, *w)
            close(y[at], want[0][-1], f"draft {j} of sequence {b}, y")
            close(r[at], want[1][-1], f"draft {j} of sequence {b}, r")
            at += 1
    path, counts, longer, after = lib.tree_accept(ints(sum(parents, [])), ints(tokens, torch.int64),
                                                  ints(choices, torch.int64), ints(lens), cu=cu(n), max_q=max(n))
    assert counts.tolist() == [len(x) for x in right] and after.tolist() == [0] * 3
    layer.accept(kv, cache, table, longer, path, counts, cu=cu(n), max_new=max(n))
    nxt = longer.tolist()
    m = [b - a for a, b in zip(lens, nxt)]
    layer(rows(lens, nxt), None, other, table, longer, cu=cu(m), max_q=max(m), max_len=64)
    if codes:     # rows do not depend on each other: the cache is as if the tokens had come as text
        for name in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"):
            assert torch.equal(getattr(cache, name), getattr(other, name)), name
    lens = nxt
    nxt = [x + 5 for x in lens]                              # and the text goes on
    got = layer(rows(lens, nxt), None, cache, table, ints(nxt), cu=cu([5] * 3), max_q=5, max_len=64)
    check(got, lens, nxt, "after the drafts")


def test_norms_without_a_rotation_and_biases_with_one(lib):
    """Head norms alone, and rotary positions next to linear biases, take the same way."""
    from mixed_precision_quantized_int8_amd.decoder import Int8DecoderLayer

    p, g = parts(8), torch.Generator().manual_seed(9)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    x = torch.randn((30, HIDDEN), generator=g).half()
    table, lens, cu = ints([[1, 0]]), ints([30]), ints([0, 30])
    outs = []
    for kw in (dict(q_norm=w), dict(rotary=lib.rotary(0), q_norm=w),
               dict(rotary=lib.rotary(D), alibi=[2.0 ** -(i + 1) for i in range(HEADS)])):
        layer = Int8DecoderLayer(*p, heads=HEADS, kv_heads=KV, **kw)
        cache = lib.new_cache(2, 1, KV, D, page_size=16)
        outs.append(layer(x.cuda(), None, cache, table, lens, cu=cu)[0])
    assert torch.equal(outs[0], outs[1])
    assert bool(outs[2].isfinite().all()) and not torch.equal(outs[2], outs[0])
    close(outs[0], reference(p, x, torch.zeros(0), False, w, None)[0], "norm of the queries alone")


@pytest.mark.parametrize("draft", [False, True])
def test_rows_behind_the_sequences(lib, monkeypatch, draft):
    """What memory held where attention answers nothing (rows behind the last sequence,
    drafts past max_q) is not seen by the product after it, whose outlier columns are those
    of all of its rows."""
    import mixed_precision_quantized_int8_amd.decoder as decoder

    p, g = parts(10), torch.Generator().manual_seed(11)
    layer = decoder.Int8DecoderLayer(*p, heads=HEADS, kv_heads=KV, rotary=lib.rotary(D))
    n, lens = [5, 3], ints([20, 9])
    table, cu = ints([[0, 1], [3, 2]]), ints([0, 5, 8])
    x = torch.randn((12, HIDDEN), generator=g).half().cuda()
    positions, masks = lib.tree_plan(ints([-1, 0, 0, 1, 2, -1, 0, 1, 0, 0, 0, 0]), lens, cu=cu, max_q=5)
    positions[8:] = 0                                        # (as the plan left them)
    name = "tree_attention" if draft else "cache_attention"
    attention, outs = getattr(decoder, name), []
    for held in (0.0, 1000.0):
        def filled(q, *a, out=None, **kw):
            out = torch.full(q.shape, held, dtype=q.dtype, device=q.device) if out is None else out
            return attention(q, *a, out=out, **kw)

        monkeypatch.setattr(decoder, name, filled)
        cache = lib.new_cache(4, 2, KV, D, page_size=16)
        for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail):
            t.zero_()
        if draft:
            outs.append(layer.draft(x, None, cache, table, lens, positions, masks, cu, max_q=4, max_len=32)[:2])
        else:
            outs.append(layer(x, None, cache, table, lens, cu, max_q=5, max_len=32))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
