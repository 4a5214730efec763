"""Cases of the operators for positions and drafts: the norm and rotary rotation of
query and key heads with its gradient, keys appended to the 8-bit cache with norm and
rotation on the way, attention for a tree of drafted tokens over that cache, and the
tree's positions, masks and accepted path.

With ``own`` false, ``run`` computes them in elementary torch operations in 32
bits (angles in 64); with ``own`` true it calls mixed_precision_quantized_int8_amd.

Layouts (the package's own):
  q [rows][q_heads][D], k, v [rows][kv_heads][D]: views of a packed projection
    [rows][q_heads + 2 kv_heads][D];
  freqs fp32 [R / 2]: token at position p turns pair i by p * freqs[i]; pair i is
    elements (i, i + R / 2), interleaved (2 i, 2 i + 1); elements from R on stay;
  cache: k_codes int8 [pages][heads][P][D], v_codes int8 [pages][heads][D][P],
    k_scale, v_scale fp32 [pages][heads] (value = code * scale); the tokens of
    a sequence's last, incomplete page are kept unquantized in k_tail
    [slots][heads][P][D] and v_tail [slots][heads][D][P];
  page_table int32 [B][pages per sequence], lengths int32 [B], slots int32 [B],
    cu int32 [B+1] (first row of each sequence in a packed tensor);
  parents int32 [rows]: the draft that a draft follows, counted within its
    sequence (-1: it follows the cached text); masks int64 [rows][words]: bit i of
    word w says that the row sees draft 64 w + i of its sequence.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6


def _case(name, op, **kw):
    return {"name": name, "op": op, **kw}


def listed():
    return [
        # one new token of a decoder layer, 32 query heads on 8, norms on both (latency)
        _case("rotate_1x40", "rotate", T=1, H=8, G=4, D=128, R=128, inter=False, norm=True, far=300,
              dtype="fp16"),
        # rows of a long prompt, 32 query heads on 8 (bandwidth)
        _case("rotate_8192x40", "rotate", T=8192, H=8, G=4, D=128, R=128, inter=False, norm=True,
              far=131072, dtype="bf16"),
        # the same operator in training: a small odd batch, part of the head, interleaved pairs
        _case("grad_333x20", "rotate_grad", T=333, H=5, G=3, D=80, R=32, inter=True, norm=True,
              far=2048, dtype="fp16"),
        # a training batch of 8192 tokens
        _case("grad_8192x40", "rotate_grad", T=8192, H=8, G=4, D=128, R=128, inter=False, norm=True,
              far=2048, dtype="bf16"),
        # a serving step: each of 16 sequences appends one token
        _case("append_16", "append", B=16, Q=1, L=300, H=8, G=4, D=128, P=16, R=128, inter=False,
              norm=True, dtype="fp16"),
        # chunks of prompts behind what is cached already; odd sizes, a quarter of the head turns
        _case("append_chunk_3x333", "append", B=3, Q=333, L=2001, H=5, G=3, D=80, P=32, R=20,
              inter=False, norm=False, dtype="bf16"),
        # whole prompts of several sequences
        _case("append_prompts_4x8192", "append", B=4, Q=8192, L=8192, H=8, G=4, D=128, P=64, R=128,
              inter=False, norm=True, dtype="bf16"),
        # a short context, one sequence with a tree of 26 drafts (latency)
        _case("tree_1x26", "tree", B=1, N=26, L=100, H=8, G=4, D=128, P=16, window=0, alibi=False,
              dtype="fp16"),
        # a serving batch, up to 64 drafts each over ragged contexts
        _case("tree_16x64x8192", "tree", B=16, N=64, L=8192, H=8, G=4, D=128, P=64, window=0,
              alibi=False, dtype="bf16"),
        # one long context, 112 heads of 128 with linear position biases, 16 drafts
        _case("tree_1x16x131072", "tree", B=1, N=16, L=131072, H=112, G=1, D=128, P=128, window=0,
              alibi=True, dtype="fp16"),
        # plan and verdict of one small tree (latency), and of a large batch of large trees
        _case("verify_1x26", "verify", B=1, N=26),
        _case("verify_64x256", "verify", B=64, N=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "rotate_grad", "append", "append", "tree", "tree", "tree",
                     "verify"])
    if op == "verify":
        return {"op": op, "B": _log(rng, 1, 64), "N": _log(rng, 1, 256)}
    D, dtype = rng.choice([64, 80, 96, 128, 128, 256]), rng.choice(["fp16", "bf16"])
    H, G = rng.choice([1, 2, 5, 8, 16]), rng.choice([1, 1, 2, 3, 4, 8])
    turn = {"R": rng.choice([D, D, D, D // 2, D // 4]), "inter": rng.random() < 0.4,
            "norm": rng.random() < 0.5}
    if op in ("rotate", "rotate_grad"):
        return {"op": op, "T": _log(rng, 1, min(16384, 8192 * 40 * 128 // (H * (G + 1) * D))), "H": H,
                "G": G, "D": D, **turn, "far": rng.choice([2048, 131072, 1 << 24]), "dtype": dtype}
    D, P = min(D, 128), rng.choice([16, 32, 64, 128])
    turn["R"] = min(turn["R"], D)
    if op == "append":
        B = _log(rng, 1, 32)
        Q = rng.choice([1, _log(rng, 2, max(2, 4 * 8192 * 48 * 128 // (B * H * (G + 2) * D)))])
        Q = min(Q, 8192)
        return {"op": op, "B": B, "Q": Q, "L": Q + rng.choice([0, _log(rng, 1, 1024)]), "H": H, "G": G,
                "D": D, "P": P, **turn, "dtype": dtype}
    B, N = _log(rng, 1, 32), _log(rng, 1, 128)
    L = _log(rng, 16, max(16, min(131072, 131072 * 56 // (B * H), (1 << 27) // (B * H * G * N))))
    return {"op": op, "B": B, "N": N, "L": L, "H": H, "G": G, "D": D, "P": P,
            "window": rng.choice([0, 0, 0, 256, 700]), "alibi": rng.random() < 0.3, "dtype": dtype}


def _ragged(B, n):
    """The first sequence has n, the others from a quarter of it up."""
    return [n if b == 0 else max(1, int(n * (0.25 + 0.75 * ((b * 0.6180339887) % 1.0)))) for b in range(B)]


def _counts(case):
    """(tokens held, rows of the call) of each sequence; a tree's rows are not held yet."""
    lens = _ragged(case["B"], case["L"])
    if case["op"] == "tree":
        return lens, _ragged(case["B"], case["N"])
    if case["Q"] == 1:
        return lens, [1] * case["B"]
    # chunks of prompts begin at a page (a pass then finds the tail as the pass before left it)
    new = [min(n, m) for n, m in zip(lens, _ragged(case["B"], case["Q"]))]
    return [(n - m) // case["P"] * case["P"] + m for n, m in zip(lens, new)], new


def _slopes(n):
    """Linear position bias slopes of n heads: a geometric sequence."""
    return [2.0 ** (-8.0 * (i + 1) / n) for i in range(n)]


def _freqs(R):
    return torch.tensor([10000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float32, device=DEV)


def _parents(n, r):
    """A tree of n drafts as a drafting model makes it: a root, then each draft behind one of
    the few before it."""
    return [-1] + [int(r.integers(max(0, j - 6), j)) for j in range(1, n)]


def _tree(parents):
    """(depth, seen drafts as Python sets) of each draft."""
    depth, seen = [], []
    for j, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        seen.append({j} | (seen[p] if p >= 0 else set()))
    return depth, seen


def _words(seen, words):
    out = np.zeros((len(seen), words), dtype=np.uint64)
    for j, s in enumerate(seen):
        for i in s:
            out[j, i >> 6] |= np.uint64(1 << (i & 63))
    return out.view(np.int64)


def _cache(case, g, lens):
    """A cache that holds `lens` tokens of each sequence, its pages in random order."""
    B, H, D, P, dt = len(lens), case["H"], case["D"], case["P"], TYPES[case["dtype"]]
    per = -(-max(lens) // P)
    pages = B * per

    def codes(*shape):
        out = torch.empty(shape, dtype=torch.int8, device=DEV)
        step = max(1, (1 << 28) // (H * P * D))
        for i in range(0, pages, step):   # bounded temporaries
            x = torch.randn(out[i:i + step].shape, generator=g, device=DEV)
            out[i:i + step] = x.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
        return out

    def scales():
        return (0.5 + torch.rand((pages, H), generator=g, device=DEV)) / 36.0

    order = torch.randperm(pages, generator=g, device=DEV)
    return {
        "k_codes": codes(pages, H, P, D), "v_codes": codes(pages, H, D, P),
        "k_scale": scales(), "v_scale": scales(),
        "k_tail": torch.randn((B, H, P, D), generator=g, device=DEV).to(dt),
        "v_tail": torch.randn((B, H, D, P), generator=g, device=DEV).to(dt),
    }, {
        "page_table": order.view(B, per).to(torch.int32).contiguous(),
        "lengths": _int(lens),
        "slots": torch.randperm(B, generator=g, device=DEV).to(torch.int32),
    }


def _int(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), device=DEV).to(dtype)


def _cu(counts):
    return _int(np.concatenate([[0], np.cumsum(counts)]))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if op == "verify":
        r = np.random.default_rng(int(seed))
        n = _ragged(case["B"], case["N"])
        parents, tokens, choices = [], [], []
        for m in n:
            p = _parents(m, r)
            t = r.integers(0, 50000, m)
            c = r.integers(0, 50000, m)
            for j in range(1, m):       # mostly the model chooses one of the drafts
                if r.random() < 0.7:
                    c[p[j]] = t[j]
            parents += p
            tokens.append(t)
            choices.append(c)
        lens = r.integers(1, 8192, len(n))
        return {"op": op, "parents": _int(parents), "tokens": _int(np.concatenate(tokens), torch.int64),
                "choices": _int(np.concatenate(choices), torch.int64), "lengths": _int(lens), "cu": _cu(n),
                "max_q": max(n)}
    H, G, D, dt = case["H"], case["G"], case["D"], TYPES[case["dtype"]]

    def weights():
        if not case["norm"]:
            return {"q_weight": None, "k_weight": None}
        return {"q_weight": (1.0 + 0.2 * randn(D)).to(dt), "k_weight": (1.0 + 0.2 * randn(D)).to(dt)}

    if op in ("rotate", "rotate_grad"):
        T = case["T"]
        s = {"op": op, "qkv": randn(T, H * (G + 2), D).to(dt), "heads": H * G, "kv_heads": H,
             "freqs": _freqs(case["R"]), "inter": case["inter"], **weights(),
             "positions": torch.randint(0, case["far"], (T,), generator=g, device=DEV).to(torch.int32)}
        if op == "rotate_grad":
            s |= {"dq": randn(T, H * G, D).to(dt), "dk": randn(T, H, D).to(dt)}
        return s
    lens, new = _counts(case)
    cache, where = _cache(case, g, lens)
    T, P = sum(new), case["P"]
    s = {"op": op, "cache": cache, "where": where, "qkv": randn(T, H * (G + 2), D).to(dt),
         "heads": H * G, "kv_heads": H, "cu": _cu(new), "max_new": max(new)}
    if op == "append":
        # the pages that the call touches, read back: as sequences that begin there
        first = [(n - m) // P for n, m in zip(lens, new)]
        rest = [n - f * P for n, f in zip(lens, first)]
        table = torch.stack([where["page_table"][b].roll(-f) for b, f in enumerate(first)])
        return s | {"freqs": _freqs(case["R"]), "inter": case["inter"], **weights(),
                    "touched": {"page_table": table, "lengths": _int(rest), "cu": _cu(rest),
                                "total": sum(rest), "max_len": max(rest)}}
    r = np.random.default_rng(int(seed))
    words = -(-max(new) // 64)
    masks, positions = [], []
    for n, m in zip(lens, new):
        depth, seen = _tree(_parents(m, r))
        masks.append(_words(seen, words))
        positions += [n + d for d in depth]
    return s | {"masks": _int(np.concatenate(masks), torch.int64), "positions": _int(positions),
                "max_len": max(lens), "scale": D ** -0.5, "window": case["window"],
                "alibi": torch.tensor(_slopes(H * G), dtype=torch.float32, device=DEV)
                if case["alibi"] else None}


def _split(s):
    qkv, n, h = s["qkv"], s["heads"], s["kv_heads"]
    return qkv[:, :n], qkv[:, n:n + h], qkv[:, n + h:]


# ---- the framework's operators ------------------------------------------------


def _run_own(s):
    import mixed_precision_quantized_int8_amd as pkg

    op = s["op"]
    if op == "verify":
        positions, masks = pkg.tree_plan(s["parents"], s["lengths"], cu=s["cu"], max_q=s["max_q"])
        path, counts, lengths, after = pkg.tree_accept(s["parents"], s["tokens"], s["choices"],
                                                       s["lengths"], cu=s["cu"], max_q=s["max_q"])
        return {"positions": positions, "masks": masks, "path": path, "counts": counts,
                "lengths": lengths, "next": after}
    q, k, v = _split(s)
    if op == "tree":
        where = s["where"]
        return {"out": pkg.tree_attention(q, k, v, pkg.KVCache(**s["cache"]), where["page_table"],
                                          where["lengths"], s["masks"], positions=s["positions"],
                                          cu=s["cu"], slots=where["slots"], max_q=s["max_new"],
                                          max_len=s["max_len"], scale=s["scale"], window=s["window"],
                                          alibi=s["alibi"])}
    rot = pkg.Rotary(s["freqs"], interleaved=s["inter"])
    norm = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": EPS}
    if op == "rotate":
        q, k = pkg.rotate_heads(q, s["positions"], rot, k=k, **norm)
        return {"q": q, "k": k}
    if op == "rotate_grad":
        dq, dk, dqw, dkw = pkg.rotate_heads_backward(s["dq"], s["positions"], rot, q=q, dk=s["dk"], k=k,
                                                     **norm)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    cache, where, t = pkg.KVCache(**s["cache"]), s["where"], s["touched"]
    q = pkg.cache_append(cache, k, v, where["page_table"], where["lengths"], q=q, rotary=rot, **norm,
                         cu=s["cu"], slots=where["slots"], max_new=s["max_new"])
    k, v = pkg.cache_read(cache, t["page_table"], t["lengths"], t["cu"], t["total"],
                          slots=where["slots"], max_len=t["max_len"])
    return {"q": q, "k": k, "v": v}


# ---- the plain forms: elementary torch operations in 32 bits --------------------


def _round_half_away(x):
    r = torch.trunc(x)
    return r + torch.where((x - r).abs() >= 0.5, torch.sign(x), torch.zeros_like(x))


def _codes(x, absmax):
    """Codes (as floats) of x over the given absolute maxima; 0 where that is 0."""
    inv = torch.where(absmax > 0, 127.0 / absmax, torch.zeros_like(absmax))
    return _round_half_away(x * inv).clamp_(-127.0, 127.0)


def _rows(cu, total):
    """(sequence, place in it) of each row of a packed tensor."""
    n = (cu[1:] - cu[:-1]).long()
    b = torch.repeat_interleave(torch.arange(n.numel(), device=cu.device), n, output_size=total)
    return b, torch.arange(total, device=cu.device) - cu.long()[b]


def _turn(x, positions, s, back=False):
    """x fp32 [T][heads][D] turned by its tokens' angles (``back``: the other way)."""
    angle = positions.double()[:, None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if back:
        sin = -sin
    R = 2 * s["freqs"].numel()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["inter"] else (x[..., :R // 2], x[..., R // 2:R])
    y = x.clone()
    ya, yb = a * cos - b * sin, a * sin + b * cos
    if s["inter"]:
        y[..., 0:R:2], y[..., 1:R:2] = ya, yb
    else:
        y[..., :R // 2], y[..., R // 2:R] = ya, yb
    return y


def _plain_rotate(x, w, positions, s):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w.float()
    return _turn(x, positions, s).to(s["qkv"].dtype)


def _plain_rotate_grad(dy, x, w, positions, s):
    g = _turn(dy.float(), positions, s, back=True)
    if w is None:
        return g.to(dy.dtype), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    n = x * r
    dw = (g * n).sum(dim=(0, 1))
    g = g * w.float()
    dx = r * (g - n * (g * n).mean(dim=-1, keepdim=True))
    return dx.to(dy.dtype), dw.to(dy.dtype)


def _held(s, where):
    """(K, V) fp32 [B][pages][H][P][D] of what the cache holds, the tail's tokens in the
    page that the lengths leave incomplete (before the call's own rows)."""
    c, pt = s["cache"], where["page_table"].long()
    k = c["k_codes"][pt].float() * c["k_scale"][pt][..., None, None]
    v = (c["v_codes"][pt].float() * c["v_scale"][pt][..., None, None]).transpose(-1, -2)
    slot = s["where"]["slots"].long()
    return k, v, c["k_tail"][slot].float()[:, None], c["v_tail"][slot].float().transpose(-1, -2)[:, None]


def _plain_append(s):
    q, k, v = _split(s)
    w, t = s["where"], s["touched"]
    T = q.shape[0]
    b, i = _rows(s["cu"], T)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    pos = (w["lengths"].long() - new)[b] + i
    outs = {"q": _plain_rotate(q, s["q_weight"], pos, s)}
    k = _plain_rotate(k, s["k_weight"], pos, s)
    P = s["cache"]["k_codes"].shape[2]
    rest = t["lengths"].long()
    old = (rest - new)[:, None]               # tokens of the first touched page that were there
    kc, vc, kt, vt = _held(s, t)
    at = torch.arange(kc.shape[1], device=kc.device)[None]
    bb, ii = _rows(t["cu"], t["total"])
    place = pos - (w["lengths"].long() - rest)[b]
    done = ((at < (rest // P)[:, None]) & (at >= 0))[:, :, None, None, None]
    for name, x, tail, rows in (("k", kc, kt, k), ("v", vc, vt, v)):
        x = torch.where((at == old // P)[:, :, None, None, None], tail, x)
        x[b, place // P, :, place % P] = rows.float()
        absmax = torch.where(done, x, torch.zeros_like(x)).abs().amax(dim=(3, 4), keepdim=True)
        x = torch.where(done, _codes(x, absmax) * (absmax / 127.0), x)
        outs[name] = x[bb, ii // P, :, ii % P].to(rows.dtype)
    return outs


def _plain_tree(s):
    q, k, v = _split(s)
    w = s["where"]
    kc, vc, kt, vt = _held(s, w)
    B, n_pages, H, P, D = kc.shape
    T, N = q.shape[0], s["max_new"]
    G = q.shape[1] // H
    lens = w["lengths"].long()
    at = torch.arange(n_pages, device=q.device)[None]
    last = (at == (lens // P)[:, None])[:, :, None, None, None]
    b, i = _rows(s["cu"], T)

    def keys(x, tail, rows):
        x = torch.where(last, tail, x).transpose(1, 2).reshape(B, H, n_pages * P, D)
        d = torch.zeros((B, N, H, D), dtype=torch.float32, device=q.device)
        d[b, i] = rows.float()
        return torch.cat([x, d.transpose(1, 2)], dim=2)

    def spread(x, fill):
        y = torch.full((B, N) + x.shape[1:], fill, dtype=x.dtype, device=q.device)
        y[b, i] = x
        return y

    kk, vv = keys(kc, kt, k), keys(vc, vt, v)
    qp = spread(q.float(), 0.0).view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    score = torch.matmul(qp, kk.transpose(-1, -2)).view(B, H, G, N, -1) * s["scale"]
    pos = spread(s["positions"].long(), 0)
    ctx = torch.arange(n_pages * P, device=q.device).expand(B, -1)
    back = pos[:, :, None] - torch.cat([ctx, pos], dim=1)[:, None]          # [B][N][keys]
    if s["alibi"] is not None:
        score -= s["alibi"].view(1, H, G, 1, 1) * back[:, None, None].float()
    bit = torch.arange(N, device=q.device)
    drafts = ((spread(s["masks"], 0)[:, :, bit >> 6] >> (bit & 63)) & 1).bool()
    seen = torch.cat([(ctx < lens[:, None])[:, None].expand(-1, N, -1), drafts], dim=2)
    if s["window"]:
        seen = seen & (back < s["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    norm = p.sum(dim=-1, keepdim=True)
    p /= torch.where(norm > 0, norm, torch.ones_like(norm))
    o = torch.matmul(p.view(B, H, G * N, -1), vv).view(B, H, G, N, D).permute(0, 3, 1, 2, 4)
    return {"out": o.reshape(B, N, H * G, D)[b, i].to(q.dtype)}


def _plain_verify(s):
    parents, T = s["parents"].long(), s["parents"].numel()
    b, i = _rows(s["cu"], T)
    first = s["cu"].long()[:-1]
    words = -(-s["max_q"] // 64)
    rows = torch.arange(T + 1, device=parents.device)                      # row T: before the root
    none = torch.full_like(parents, T)
    up = torch.cat([torch.where(parents >= 0, first[b] + parents, none), none[:1]])
    bit = torch.ones_like(i) << (i & 63)
    masks = torch.where(rows[:words] == (i >> 6)[:, None], bit[:, None], torch.zeros_like(bit)[:, None])
    masks = torch.cat([masks, torch.zeros_like(masks[:1])])
    depth = (up != T).long()
    # the choice of its parent names a draft, and it is the first such child; the root is known
    tokens = torch.cat([s["tokens"], s["tokens"][:1]])
    choices = torch.cat([s["choices"], s["choices"][:1]])
    hit = (tokens == choices[up]) & (up != T)
    least = torch.full_like(up, T).scatter_reduce(0, up, torch.where(hit, rows, T), "amin")
    good = (hit & (least[up] == rows)) | (rows == T)
    good[:T] |= i == 0
    for _ in range((s["max_q"] - 1).bit_length()):                         # twice the ancestors a step
        masks = masks | masks[up]
        depth = depth + depth[up]
        good = good & good[up]
        up = up[up]
    # accepted drafts are one path: its length and places
    good = good[:T].long()
    counts = torch.zeros_like(first).scatter_add(0, b, good)
    place = torch.where(good > 0, first[b] + depth[:T], none)
    path = torch.full_like(rows, -1).scatter(0, place, rows[:T])
    end = path[first + counts - 1]
    lens = s["lengths"].long()
    return {"positions": (lens[b] + depth[:T]).int(), "masks": masks[:T], "path": path[:T].int(),
            "counts": counts.int(), "lengths": (lens + counts).int(), "next": s["choices"][end]}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "verify":
        return _plain_verify(s)
    if op == "tree":
        return _plain_tree(s)
    if op == "append":
        return _plain_append(s)
    q, k, _ = _split(s)
    if op == "rotate":
        return {"q": _plain_rotate(q, s["q_weight"], s["positions"], s),
                "k": _plain_rotate(k, s["k_weight"], s["positions"], s)}
    dq, dqw = _plain_rotate_grad(s["dq"], q, s["q_weight"], s["positions"], s)
    dk, dkw = _plain_rotate_grad(s["dk"], k, s["k_weight"], s["positions"], s)
    return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


def work(case):
    op = case["op"]
    if op == "verify":
        rows = sum(_ragged(case["B"], case["N"]))
        words = -(-case["N"] // 64)
        return {"bytes": rows * (4 + 8 + 8 + 4 + 8 * words + 4) + case["B"] * 24, "flops": rows * 64}
    H, G, D = case["H"], case["G"], case["D"]
    if op in ("rotate", "rotate_grad"):
        n = case["T"] * H * (G + 1) * D
        small = 4 * case["T"] + 2 * case["R"] + (4 * D if case["norm"] else 0)
        if op == "rotate":
            return {"bytes": 4 * n + small, "flops": 7 * n}
        return {"bytes": (6 if case["norm"] else 4) * n + small + (4 * D if case["norm"] else 0),
                "flops": 14 * n}
    lens, new = _counts(case)
    T, P = sum(new), case["P"]
    if op == "append":
        # q turned; the new tokens in; the pages that the write completes and the tails out;
        # every token of a touched page read back from codes or tail
        done = [n // P - (n - m) // P for n, m in zip(lens, new)]
        written = sum(2 * m for m in new) + sum(d * (P + 4 / D) for d in done)
        written += sum(2 * min(n % P, m) for n, m in zip(lens, new))
        rest = [n - (n - m) // P * P for n, m in zip(lens, new)]
        read = sum((n - n % P) + 2 * (n % P) + 2 * n for n in rest)
        return {"bytes": 2 * H * D * (written + read) + 4 * T * H * G * D,
                "flops": T * H * D * (7 * (G + 1) + 6)}
    W = case["window"]
    keys = [min(n, W) if W else n for n in lens]
    pairs = sum(m * n + m * (m + 1) // 2 for n, m in zip(keys, new))
    return {"bytes": 2 * sum(keys) * H * D + 4 * T * H * (G + 1) * D, "flops": 4 * D * H * G * pairs}


# ---- the definitions in 64 bits -------------------------------------------------


def _exact_rotate(x, w, positions, s):
    """The definition on complex numbers: a pair is a + bi, its turn a factor exp(i t)."""
    d = torch.float64
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    h = s["freqs"].numel()
    t = positions.to(d)[:, None, None] * s["freqs"].to(d)
    turned = x[..., :2 * h]
    z = torch.view_as_complex(turned.unflatten(-1, (h, 2) if s["inter"] else (2, h))
                              .transpose(-1, -1 if s["inter"] else -2).contiguous())
    y = torch.view_as_real(z * torch.polar(torch.ones_like(t), t))
    y = (y if s["inter"] else y.transpose(-1, -2)).flatten(-2)
    return torch.cat([y, x[..., 2 * h:]], dim=-1)


def _exact_page(x):
    top = x.abs().amax(dim=(1, 3), keepdim=True)
    c = x * (127.0 / torch.where(top > 0, top, torch.ones_like(top)))
    return torch.sign(c) * torch.floor(c.abs() + 0.5) * top / 127.0


def _exact_verify(s):
    parents, tokens, choices = s["parents"].tolist(), s["tokens"].tolist(), s["choices"].tolist()
    cu, lens = s["cu"].tolist(), s["lengths"].tolist()
    words = -(-s["max_q"] // 64)
    positions, masks, path, counts, after = [], [], [], [], []
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        depth, seen = _tree(parents[lo:hi])
        positions += [n + d for d in depth]
        masks.append(_words(seen, words))
        got = [0]
        while True:
            follow = [j for j in range(hi - lo)
                      if parents[lo + j] == got[-1] and tokens[lo + j] == choices[lo + got[-1]]]
            if not follow:
                break
            got.append(follow[0])
        path += [lo + j for j in got] + [-1] * (hi - lo - len(got))
        counts.append(len(got))
        after.append(choices[lo + got[-1]])
    return {"positions": _int(positions), "masks": _int(np.concatenate(masks), torch.int64),
            "path": _int(path), "counts": _int(counts),
            "lengths": _int([n + m for n, m in zip(lens, counts)]), "next": _int(after, torch.int64)}


def exact(case, seed):
    s = prepare(case, seed)
    d, op = torch.float64, case["op"]
    if op == "verify":
        return _exact_verify(s)
    q, k, v = (x.to(d) for x in _split(s))
    if op in ("rotate", "rotate_grad"):
        out = {}
        for name, x, dy in (("q", q, s.get("dq")), ("k", k, s.get("dk"))):
            w = s[name + "_weight"]
            w = None if w is None else w.to(d)
            if op == "rotate":
                out[name] = _exact_rotate(x, w, s["positions"], s)
                continue
            x = x.clone().requires_grad_()
            if w is not None:
                w.requires_grad_()
            _exact_rotate(x, w, s["positions"], s).backward(dy.to(d))
            out["d" + name] = x.grad
            out["d" + name + "w"] = None if w is None else w.grad
        return {n: out[n] for n in (("q", "k") if op == "rotate" else ("dq", "dk", "dqw", "dkw"))}
    c, where = s["cache"], s["where"]
    lens, cu = where["lengths"].tolist(), s["cu"].tolist()
    H, D, P, G = case["H"], case["D"], case["P"], case["G"]

    def held(b, lo, n):
        """Keys and values [n - lo][H][D] of tokens lo .. n - 1 of sequence b (lo: a page's first)."""
        full, slot = n // P, int(where["slots"][b])
        pages = where["page_table"][b, lo // P:full].long()
        kk = c["k_codes"][pages].to(d) * c["k_scale"][pages].to(d)[:, :, None, None]
        vv = c["v_codes"][pages].to(d) * c["v_scale"][pages].to(d)[:, :, None, None]
        kk = kk.permute(0, 2, 1, 3).reshape(-1, H, D)
        vv = vv.permute(0, 3, 1, 2).reshape(-1, H, D)
        r = n - full * P
        return (torch.cat([kk, c["k_tail"][slot, :, :r].to(d).transpose(0, 1)]),
                torch.cat([vv, c["v_tail"][slot, :, :, :r].to(d).permute(2, 0, 1)]))

    if op == "append":
        dt = s["qkv"].dtype
        pos = torch.cat([torch.arange(n - (cu[b + 1] - cu[b]), n, device=DEV) for b, n in enumerate(lens)])
        qw, kw = (None if s[x] is None else s[x].to(d) for x in ("q_weight", "k_weight"))
        # keys are kept as 16-bit tokens until their page is complete: rounded here
        k = _exact_rotate(k, kw, pos, s).to(dt).to(d)
        outs = [[], []]
        for b, n in enumerate(lens):
            old = n - (cu[b + 1] - cu[b])
            lo, hi = old // P * P, n // P * P
            for j, (x, rows) in enumerate(zip(held(b, lo, old), (k, v))):
                x = torch.cat([x, rows[cu[b]:cu[b + 1]]])
                m = max(hi - lo, 0)
                outs[j].append(torch.cat([_exact_page(x[:m].view(-1, P, H, D)).view(-1, H, D), x[m:]])
                               if m else x)
        return {"q": _exact_rotate(q, qw, pos, s), "k": torch.cat(outs[0]), "v": torch.cat(outs[1])}
    got = []
    for b, n in enumerate(lens):
        kk, vv = (torch.cat([x, y[cu[b]:cu[b + 1]]]) for x, y in zip(held(b, 0, n), (k, v)))
        m = cu[b + 1] - cu[b]
        bits = s["masks"][cu[b]:cu[b + 1]].cpu().numpy().view(np.uint64)
        drafts = torch.tensor([[bool(int(bits[j, i >> 6]) >> (i & 63) & 1) for i in range(m)]
                               for j in range(m)], device=DEV)
        at = s["positions"][cu[b]:cu[b + 1]].long()
        back = at[:, None] - torch.cat([torch.arange(n, device=DEV), at])[None]
        hide = torch.cat([torch.zeros((m, n), dtype=torch.bool, device=DEV), ~drafts], dim=1)
        if case["window"]:
            hide |= back >= case["window"]
        o = torch.empty((m, H, G, D), dtype=d, device=DEV)
        qq = q[cu[b]:cu[b + 1]].view(m, H, G, D)
        for h in range(H):
            a = (qq[:, h].reshape(m * G, D) @ kk[:, h].T).view(m, G, n + m) * s["scale"]
            if s["alibi"] is not None:
                a -= s["alibi"].to(d)[h * G:(h + 1) * G].view(1, G, 1) * back[:, None]
            a = torch.softmax(a.masked_fill(hide[:, None], -math.inf), dim=-1)
            o[:, h] = (a.view(m * G, n + m) @ vv[:, h]).view(m, G, D)
        got.append(o.view(m, H * G, D))
    return {"out": torch.cat(got)}
