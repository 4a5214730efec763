"""The 8-bit decoder layer (decoder.py) on the GPU: prompts, then single tokens, over
one paged cache, against the same layer in float64 on the unquantized weights."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(i8l):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return i8l


HIDDEN, HEADS, KV, D, FFN = 256, 8, 2, 64, 768


def parts(seed):
    g = torch.Generator().manual_seed(seed)

    def linear(i, o, bias=True):
        lin = torch.nn.Linear(i, o, bias=bias)
        with torch.no_grad():
            lin.weight.copy_(torch.randn((o, i), generator=g) * i ** -0.5)
            if bias:
                lin.bias.copy_(torch.randn(o, generator=g) * 0.1)
        return lin

    norms = [(1 + 0.1 * torch.randn(HIDDEN, generator=g)) for _ in range(2)]
    return (norms[0], linear(HIDDEN, (HEADS + 2 * KV) * D), linear(HEADS * D, HIDDEN), norms[1],
            linear(HIDDEN, FFN), linear(FFN, HIDDEN, bias=False))


def reference(p, x, alibi):
    """(y, r') of one whole sequence in float64."""
    norm1, qkv, out, norm2, up, down = p
    f = lambda lin, v: v @ lin.weight.detach().double().T + (0 if lin.bias is None else  # noqa: E731
                                                            lin.bias.detach().double())
    norm = lambda v, w: v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5) * w.double()  # noqa: E731
    r = x.double()
    n = r.shape[0]
    z = f(qkv, norm(r, norm1)).view(n, HEADS + 2 * KV, D)
    back = (torch.arange(n)[:, None] - torch.arange(n)[None]).double()
    o = torch.empty((n, HEADS, D), dtype=torch.float64)
    for h in range(HEADS):
        kv = h // (HEADS // KV)
        s = z[:, h] @ z[:, HEADS + kv].T * D ** -0.5
        if alibi is not None:
            s = s - alibi[h] * back
        o[:, h] = torch.softmax(s.masked_fill(back < 0, -math.inf), 1) @ z[:, HEADS + KV + kv]
    r = r + f(out, o.view(n, HEADS * D))
    return f(down, torch.nn.functional.gelu(f(up, norm(r, norm2)))), r


@pytest.mark.parametrize("use_alibi", [False, True])
def test_prompts_then_tokens(lib, use_alibi):
    from mixed_precision_quantized_int8_amd.decoder import Int8DecoderLayer

    print("decoder layer, alibi", use_alibi, flush=True)
    p = parts(3)
    alibi = [2.0 ** -(i + 1) for i in range(HEADS)] if use_alibi else None
    layer = Int8DecoderLayer(*p, heads=HEADS, kv_heads=KV, alibi=alibi)
    g = torch.Generator().manual_seed(4)
    total, prompt = [75, 48, 16], [60, 33, 1]
    x = [torch.randn((n, HIDDEN), generator=g).half() for n in total]
    B, P = 3, 16
    per = -(-max(total) // P)
    cache = lib.new_cache(B * per, B, KV, D, page_size=P)
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    got_y, got_r = [[] for _ in x], [[] for _ in x]

    def run(lo, hi, one):
        rows = torch.cat([s[a:b] for s, a, b in zip(x, lo, hi)]).cuda()
        n = [b - a for a, b in zip(lo, hi)]
        cu = None if one else torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32, device="cuda")
        y, r = layer(rows, None, cache, table, torch.tensor(hi, dtype=torch.int32, device="cuda"),
                     cu=cu, max_q=max(n), max_len=max(total))
        at = 0
        for b in range(B):
            got_y[b].append(y[at:at + n[b]].cpu().double())
            got_r[b].append(r[at:at + n[b]].cpu().double())
            at += n[b]

    run([0] * B, prompt, False)
    run(prompt, [n + 7 for n in prompt], False)          # a second chunk of each
    at = [n + 7 for n in prompt]
    for _ in range(8):                                   # then a token at a time
        run(at, [n + 1 for n in at], True)
        at = [n + 1 for n in at]
    assert at == total
    for b in range(B):
        y, r = reference(p, x[b], alibi)
        for name, got, want in (("y", got_y[b], y), ("r", got_r[b], r)):
            got = torch.cat(got)
            assert got.shape == want.shape
            # Each 8-bit operand is within half a step of absmax / 127, about 1 % of a
            # normal row's rms (absmax ~ 3.3 rms: 0.5 / 127 * 3.3 = 1.3 %, uniform: / sqrt 3).
            # A product of two such operands errs by 1.1 % of its rms; four of them in a
            # row, and the cache's two, stay below 3 % together (errors add in squares).
            rel = float((got - want).norm() / want.norm())
            assert rel < 0.03, f"{name} of sequence {b}: {rel:.4f}"


def test_layer_refuses_sizes_that_do_not_fit(lib):
    from mixed_precision_quantized_int8_amd.decoder import Int8DecoderLayer

    p = parts(5)
    with pytest.raises(ValueError, match="heads"):
        Int8DecoderLayer(*p, heads=7, kv_heads=2)
    with pytest.raises(ValueError, match="fit"):
        Int8DecoderLayer(p[0], p[1], p[4], p[3], p[4], p[5], heads=HEADS, kv_heads=KV)
