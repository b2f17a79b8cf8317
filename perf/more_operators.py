"""The operators of a step of decoding with trees of drafted tokens, around block-sparse attention: cases, plain forms and exact results.

Five operators that a server calls next to the cache, attention and verification calls:

  rope      Q and K are (normalised and) rotated to their positions, Q is quantised for the attention, K and V are written into their pages
  mask      a batch's trees of drafted tokens, given by parents, become ancestor masks and positions
  attend    dense attention of those tokens over the paged cache: the whole context, and of the tree the ancestors alone
  accept    the path of the tree that the target's own tokens follow, and its rows of every layer's cache moved to their place in the sequence
  logprobs  log probabilities of given tokens with their ranks, the rows' entropies and best alternatives

``own`` chooses between the plain forms (elementary torch operations) and this package's calls.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE, D = 128, 128
E4M3_MAX, E2M1_MAX = 448.0, 6.0
SLOT = 9216  # bytes of an NVFP4 K or V slot: 128 x 64 of codes, 128 x 8 block scales
MOST_NODES = 256  # tokens of a tree
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    return [
        # one step of 64 requests with 8 drafted tokens each, half of each head rotated, Q and K normalised (latency)
        {"name": "rope decode 64x8", "op": "rope", "fmt": "e4m3", "type": "bf16", "hq": 16, "heads": 2, "B": 64, "q_lo": 8, "q_hi": 8, "ctx": 4096,
         "rot": 64, "interleaved": False, "axes": 1, "far": 0, "norm": True, "q8": True, "lens": 1},
        # a large prefill batch, whole heads rotated, far behind the start of a long stream (bandwidth)
        {"name": "rope prefill 8 x 8k", "op": "rope", "fmt": "e4m3", "type": "bf16", "hq": 32, "heads": 4, "B": 8, "q_lo": 7001, "q_hi": 8192, "ctx": 9000,
         "rot": 128, "interleaved": False, "axes": 1, "far": 900000, "norm": False, "q8": True, "lens": 2},
        # image and video tokens with positions of three axes, neighbouring pairs, into NVFP4 pages, Q for the bf16 kernel
        {"name": "rope nvfp4 3 axes", "op": "rope", "fmt": "nvfp4", "type": "fp16", "hq": 16, "heads": 2, "B": 5, "q_lo": 129, "q_hi": 4096, "ctx": 5000,
         "rot": 96, "interleaved": True, "axes": 3, "far": 0, "norm": True, "q8": False, "lens": 3},
        # one small tree (latency)
        {"name": "mask 1x16", "op": "mask", "B": 1, "q_lo": 16, "q_hi": 16, "ctx": 5000, "lens": 4},
        # the largest trees of a large batch, ragged
        {"name": "mask 256x255", "op": "mask", "B": 256, "q_lo": 100, "q_hi": 255, "ctx": 100000, "lens": 5},
        # small trees of a few requests over contexts of their own (latency)
        {"name": "attend 4x16 own 16k", "op": "attend", "hq": 16, "heads": 2, "B": 4, "q_lo": 16, "q_hi": 16, "prefix": 0, "own_lo": 8000, "own_hi": 16384, "lens": 6},
        # trees of up to 64 tokens for 32 requests behind a 32k-token shared document
        {"name": "attend 32x64 over 32k", "op": "attend", "hq": 16, "heads": 2, "B": 32, "q_lo": 33, "q_hi": 64, "prefix": 256, "own_lo": 64, "own_hi": 3000, "lens": 7},
        # nothing shared: 16 requests of up to 128k tokens, trees of 24
        {"name": "attend 16x24 own 128k", "op": "attend", "hq": 16, "heads": 2, "B": 16, "q_lo": 24, "q_hi": 24, "prefix": 0, "own_lo": 32768, "own_hi": 131072, "lens": 8},
        # one request, a small tree, four layers (latency)
        {"name": "accept 1x16, 4 layers", "op": "accept", "fmt": "e4m3", "heads": 2, "layers": 4, "B": 1, "q_lo": 16, "q_hi": 16, "ctx": 1000, "lens": 9},
        # 64 requests, trees of up to 64, 32 layers in one call
        {"name": "accept 64x64, 32 layers", "op": "accept", "fmt": "e4m3", "heads": 2, "layers": 32, "B": 64, "q_lo": 40, "q_hi": 64, "ctx": 160, "lens": 10},
        # the answer's log probabilities of a decode step, an odd vocabulary, twenty alternatives (few rows)
        {"name": "logprobs 16 of 200k", "op": "logprobs", "type": "fp32", "T": 16, "V": 200003, "top": 20},
        # a prompt's log probabilities
        {"name": "logprobs 2048 of 131k", "op": "logprobs", "type": "bf16", "T": 2048, "V": 131072, "top": 5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "rope", "mask", "attend", "attend", "accept", "logprobs", "logprobs"))
    lens = rng.randrange(1, 1 << 20)
    if op == "rope":
        heads, group = rng.choice(((1, 1), (1, 16), (2, 8), (3, 5), (4, 8), (8, 2)))
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 1200000 // (B * heads * (group + 2))))  # rows of a head: their bytes below the largest case's in any type
        return {"op": op, "fmt": rng.choice(("e4m3", "e4m3", "nvfp4")), "type": rng.choice(tuple(TYPES)), "hq": heads * group, "heads": heads, "B": B,
                "q_lo": rng.randint(1, hi), "q_hi": hi, "ctx": hi + _log(rng, 1, 2000), "rot": rng.choice((2, 20, 32, 64, 64, 80, 96, 128, 128)),
                "interleaved": rng.random() < 0.4, "axes": rng.choice((1, 1, 3)), "far": rng.choice((0, 0, 100003, 1000000)), "norm": rng.random() < 0.5,
                "q8": rng.random() < 0.6, "lens": lens}
    if op == "mask":
        hi = _log(rng, 1, MOST_NODES)
        return {"op": op, "B": _log(rng, 1, 65280 // hi), "q_lo": rng.randint(1, hi), "q_hi": hi, "ctx": _log(rng, hi, 200000), "lens": lens}
    if op == "attend":
        heads, group = rng.choice(((1, 1), (1, 16), (2, 4), (2, 8), (4, 3), (8, 4)))
        hi = rng.choice((1, 8, _log(rng, 9, 64), _log(rng, 9, MOST_NODES)))
        B = _log(rng, 1, max(1, min(32, 32768 // (heads * group * hi))))
        most = max(4, min(1024, 2 ** 22 // (B * heads * group * hi)))  # pages: rows x keys below the largest case's
        prefix = rng.choice((0, _log(rng, 1, most), _log(rng, 1, most)))
        own_hi = hi + _log(rng, 1, PAGE * (min(most, 32) if prefix else most))
        return {"op": op, "hq": heads * group, "heads": heads, "B": B, "q_lo": rng.randint(1, hi), "q_hi": hi, "prefix": prefix,
                "own_lo": rng.randint(hi, own_hi), "own_hi": own_hi, "lens": lens}
    if op == "accept":
        hi, heads, layers = _log(rng, 1, MOST_NODES), rng.choice((1, 2, 3, 4, 8)), _log(rng, 1, 32)
        B = _log(rng, 1, max(1, min(64, 600000 // (layers * heads * (hi + 200)))))
        return {"op": op, "fmt": rng.choice(("e4m3", "nvfp4")), "heads": heads, "layers": layers, "B": B, "q_lo": rng.randint(1, hi), "q_hi": hi,
                "ctx": hi + _log(rng, 1, 200), "lens": lens}
    V = _log(rng, 500, 200003)
    return {"op": op, "type": rng.choice(tuple(TYPES)), "T": _log(rng, 1, min(4096, 2 ** 27 // V)), "V": V, "top": rng.choice((0, 1, 5, 20, 32))}


# --------------------------------------------------------------------------- inputs


def _lengths(case):
    """Per request: its new tokens, and its length with them (they are its last tokens)."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    if case["op"] == "attend":
        q[0] = case["q_hi"]
        return q, [case["prefix"] * PAGE + max(n, r.randint(case["own_lo"], case["own_hi"])) for n in q]
    return q, [r.randint(n, max(n, case["ctx"])) for n in q]


def _cum(v, dev):
    return torch.tensor([0] + [sum(v[:i + 1]) for i in range(len(v))], dtype=torch.int32, device=dev)


def _normal(shape, g, dev, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=dev, dtype=dtype)


def _float32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def _pool(pages, heads, g, dev):
    """An E4M3 pool of N(0, 1) keys and values with one scale each for K and V."""
    out = torch.empty((pages, heads, PAGE, 2 * D), dtype=torch.float8_e4m3fn, device=dev)
    scale = _float32(5.7139 / E4M3_MAX)
    step = max(1, (1 << 26) // (heads * PAGE * 2 * D))
    for a in range(0, pages, step):
        x = _normal((min(step, pages - a), heads, PAGE, 2 * D), g, dev)
        out[a:a + step] = (x / scale).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return out, scale


def _pool4(pages, heads, g, dev):
    """An NVFP4 pool of random codes with block scales of the size that N(0, 1) values get under the global scale."""
    out = torch.empty((pages, heads, 2, SLOT), dtype=torch.uint8, device=dev)
    out[..., :PAGE * 64] = torch.randint(0, 256, (pages, heads, 2, PAGE * 64), generator=g, device=dev, dtype=torch.uint8)
    s = torch.rand((pages, heads, 2, PAGE * 8), generator=g, device=dev) * 30 + 10
    out[..., PAGE * 64:] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return out, _float32(5.1377 / E4M3_MAX)


def _table(seq, shared, spare, r, dev):
    """A block table over a permuted pool in which all rows begin with the same `shared` pages; the pool has `spare` pages that nothing uses."""
    pages = [-(-s // PAGE) for s in seq]
    total = shared + sum(p - shared for p in pages) + spare
    perm = torch.from_numpy(np.random.RandomState(r).permutation(total).astype("int32"))
    table = torch.full((len(seq), max(max(pages), 1)), -1, dtype=torch.int32)
    at = shared
    for b, p in enumerate(pages):
        table[b, :shared] = perm[:shared]
        table[b, shared:p] = perm[at:at + p - shared]
        at += p - shared
    return table.to(dev), total


def _places(s):
    """(request, index in the request) of every new token."""
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    return b, t - s["cu_q"].long()[b]


def _tree(s, g):
    """Parents of random trees, of each request's tokens by their index in it: the first is the root."""
    _, i = _places(s)
    u = torch.rand((s["T"],), generator=g, device="cuda", dtype=torch.float64)
    # half of the tokens follow one of the last eight before them, so that trees are as deep as they are broad
    near = torch.rand((s["T"],), generator=g, device="cuda") < 0.5
    lo = torch.where(near, (i - 8).clamp(min=0), torch.zeros_like(i))
    return torch.where(i > 0, lo + (u * (i - lo)).long(), torch.full_like(i, -1)).to(torch.int32)


def _padded(s, flat, fill):
    """Values of the tokens [T] as [B, most of a request], `fill` behind a request's last."""
    b, i = _places(s)
    out = torch.full((s["case"]["B"], s["max_q"]), fill, dtype=flat.dtype, device="cuda")
    out[b, i] = flat
    return out


def _ancestors(s):
    """[B, n, n] booleans: whether the second node is the first or one of its ancestors."""
    p = _padded(s, s["parents"].long(), -1)
    n = p.shape[1]
    at = torch.arange(n, device="cuda")
    up = (p[..., None] == at) | (at[:, None] == at)
    for _ in range((n - 1).bit_length()):  # paths of up to 2, 4, 8, ... steps
        up = torch.matmul(up.float(), up.float()) > 0
    return up


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] == "logprobs":
        T, V, t = case["T"], case["V"], TYPES[case["type"]]
        s["logits"] = torch.empty((T, V), dtype=t, device=dev)
        step = max(1, (1 << 26) // V)
        for a in range(0, T, step):  # peaked, as language models give them
            s["logits"][a:a + step] = (3 * _normal((min(step, T - a), V), g, dev)).to(t)
        # half of the tokens are likely ones, as a sampler takes them, half any, as a prompt has them
        like = (s["logits"][:, :64].float()).argmax(-1)
        some = torch.randint(0, V, (T,), generator=g, device=dev)
        s["tokens"] = torch.where(torch.rand((T,), generator=g, device=dev) < 0.5, like, some).to(torch.int32)
        return s
    q, seq = _lengths(case)
    s["cu_q"], s["cu_k"], s["T"] = _cum(q, dev), _cum(seq, dev), sum(q)
    s["max_q"], s["max_k"] = max(q), max(seq)
    b, i = _places(s)
    s["first"] = s["cu_k"].diff() - s["cu_q"].diff()  # a request's tokens in the cache before these
    if case["op"] == "mask":
        s["parents"] = _tree(s, g)
        return s
    if case["op"] == "rope":
        s["table"], pages = _table(seq, 0, 3, seed % (1 << 31), dev)
        s["kv"], scale = (_pool4 if case["fmt"] == "nvfp4" else _pool)(pages, case["heads"], g, dev)
        s["k_scale"], s["v_scale"] = scale, _float32(scale * 1.2345)
        s["q_scale"] = _float32(5.9021 / E4M3_MAX) if case["q8"] else None
        s["dtype"], hq, heads = TYPES[case["type"]], case["hq"], case["heads"]
        # Q, K and V as a fused projection leaves them: parts of one row a token
        x = _normal((s["T"], hq + 2 * heads, D), g, dev).to(s["dtype"])
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + heads], x[:, hq + heads:]
        s["inv_freq"] = 5e6 ** -(torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
        s["inv_freq_here"] = s["inv_freq"].to(dev)
        pos = s["first"].long()[b] + i // 2 + case["far"]  # as a tree's tokens have them
        if case["axes"] == 1:
            s["axes"], s["positions"] = None, pos.to(torch.int32)
        else:  # time, height, width: a third of the frequencies each, in turn
            s["axes"] = [j % 3 for j in range(case["rot"] // 2)]
            s["positions"] = torch.stack((pos, pos + i % 37, pos + i // 37 % 23)).to(torch.int32)
        w = 1 + 0.2 * _normal((2, D), g, dev)
        s["q_norm"], s["k_norm"] = (w[0].contiguous(), w[1].contiguous()) if case["norm"] else (None, None)
        if own:
            import block_sparse_attention_prefill_gb300 as msa

            s["rope"] = msa.MsaRope(s["inv_freq"], interleaved=case["interleaved"], axes=s["axes"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return s
    s["parents"] = _tree(s, g)
    if case["op"] == "attend":
        s["table"], pages = _table(seq, case["prefix"], 2, seed % (1 << 31), dev)
        s["kv"], s["k_scale"] = _pool(pages, case["heads"], g, dev)
        s["v_scale"] = s["k_scale"]
        s["q_scale"] = _float32(5.7139 / E4M3_MAX)
        x = _normal((s["T"], case["hq"], D), g, dev)
        s["q"] = (x / s["q_scale"]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["softmax_scale"], s["prefix"] = 1.0 / math.sqrt(D), case["prefix"]
        s["mask"] = _words(_ancestors(s), s)  # kept for all layers of a step
        return s
    s["table"], pages = _table(seq, 0, 3, seed % (1 << 31), dev)
    make = _pool4 if case["fmt"] == "nvfp4" else _pool
    s["kv"] = [make(pages, case["heads"], g, dev)[0] for _ in range(case["layers"])]
    s["drafts"] = torch.randint(0, 50000, (s["T"],), generator=g, device=dev, dtype=torch.int32)
    # the target agrees with one of a token's children (the last, if it has any) four times of five
    last = torch.full((s["T"],), -1, dtype=torch.long, device=dev)
    up = (s["cu_q"].long()[b] + s["parents"].long()).clamp(min=0)
    t = torch.arange(s["T"], device=dev)
    last.scatter_reduce_(0, up[i > 0], t[i > 0], "amax")
    agree = (last >= 0) & (torch.rand((s["T"],), generator=g, device=dev) < 0.8)
    other = torch.randint(0, 50000, (s["T"],), generator=g, device=dev, dtype=torch.int32)
    s["chosen"] = torch.where(agree, s["drafts"][last.clamp(min=0)], other)
    return s


# --------------------------------------------------------------------------- plain forms


def _encode4(x, g):
    """fp32 [..., 128] -> E2M1 codes [..., 64] (two a byte, the first in the low nibble) and E4M3 block scales [..., 8]."""
    xb = x.reshape(*x.shape[:-1], 8, 16)
    scale = (xb.abs().amax(-1) / (E2M1_MAX * g)).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    den = (scale.float() * g).unsqueeze(-1)
    y = torch.where(den > 0, xb / den, torch.zeros_like(xb))
    grid = torch.tensor(E2M1, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = y.abs().clamp(max=E2M1_MAX)
    low = torch.bucketize(a, mid)  # the middle itself goes to the lower neighbour ...
    high = torch.bucketize(a, mid, right=True)  # ... or to the upper one: the even of the two is taken
    code = torch.where(low % 2 == 0, low, high)
    code = (code | ((y < 0) & (code > 0)).long() << 3).reshape(x.shape).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def _decode4(codes, scales):
    """Codes [..., 64] and E4M3 scales [..., 8] -> the E4M3 values that the attention reads, [..., 128]."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = grid[torch.stack((codes & 15, codes >> 4), -1).long()].reshape(*codes.shape[:-1], 8, 16) * scales.float().unsqueeze(-1)
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).reshape(*codes.shape[:-1], D)


def _values4(kv):
    """A whole NVFP4 pool as the E4M3 pool that the attention reads."""
    n, h = kv.shape[:2]
    halves = [_decode4(kv[:, :, j, :PAGE * 64].reshape(n, h, PAGE, 64), kv[:, :, j, PAGE * 64:].reshape(n, h, PAGE, 8).view(torch.float8_e4m3fn)) for j in (0, 1)]
    return torch.cat([x.view(torch.uint8) for x in halves], -1).view(torch.float8_e4m3fn)


def _rotated(s, x, weight, type_):
    """Rows [T, heads, 128] normalised and rotated, in `type_` with angles in 64 bits."""
    case, half = s["case"], s["case"]["rot"] // 2
    x = x.to(type_)
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.to(type_)
    pos = s["positions"].double().reshape(case["axes"], -1)
    of = torch.zeros(half, dtype=torch.long) if s["axes"] is None else torch.tensor(s["axes"])
    angle = pos[of.to(pos.device)].T * s["inv_freq_here"]  # [T, half]
    cos, sin = angle.cos().to(type_)[:, None], angle.sin().to(type_)[:, None]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if case["interleaved"] else (x[..., :half], x[..., half:2 * half])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.stack(y, -1).flatten(-2) if case["interleaved"] else torch.cat(y, -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _rows(s):
    """Page and row in the page of every new token."""
    b, i = _places(s)
    pos = s["first"].long()[b] + i
    return s["table"].long()[b, pos // PAGE], pos % PAGE


def _plain_rope(s):
    page, row = _rows(s)
    q, kv = _rotated(s, s["q"], s["q_norm"], torch.float32), s["kv"]
    k = _rotated(s, s["k"], s["k_norm"], torch.float32)
    for half, x, g in ((0, k, s["k_scale"]), (1, s["v"].float(), s["v_scale"])):
        if s["case"]["fmt"] == "e4m3":
            code = (x / g).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            kv.view(torch.uint8)[page, :, row, half * D:(half + 1) * D] = code.view(torch.uint8)
        else:
            codes, scale = _encode4(x, g)
            kv[:, :, half, :PAGE * 64].view(*kv.shape[:2], PAGE, 64)[page, :, row] = codes
            kv[:, :, half, PAGE * 64:].view(*kv.shape[:2], PAGE, 8)[page, :, row] = scale.view(torch.uint8)
    q = (q / s["q_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) if s["case"]["q8"] else q.to(torch.bfloat16)
    return [q, kv if s["case"]["fmt"] == "e4m3" else _values4(kv)]


def _words(up, s):
    """Booleans [B, n, n] as the tokens' mask words, int32 [T, ceil(n / 32)], the first node in the lowest bit."""
    n = up.shape[-1]
    bits = torch.nn.functional.pad(up, (0, -n % 32)).view(*up.shape[:2], -1, 32).long()
    w = (bits << torch.arange(32, device="cuda")).sum(-1)
    b, i = _places(s)
    w = w[b, i]
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _plain_mask(s):
    up = _ancestors(s)
    b, i = _places(s)
    depth = up.sum(-1) - 1
    return [_words(up, s), (s["first"].long()[b] + depth[b, i]).to(torch.int32)]


def _plain_attend(s):
    case, P = s["case"], s["prefix"]
    B, H, G, n = case["B"], case["heads"], case["hq"] // case["heads"], s["max_q"]
    dev = s["q"].device
    b, i = _places(s)
    # queries padded to the largest tree, [H, B, n, G, D]
    q = torch.zeros((B, n, H, G, D), device=dev)
    q[b, i] = s["q"].float().view(-1, H, G, D)
    q = q.permute(2, 0, 1, 3, 4) * (s["q_scale"] * s["k_scale"] * s["softmax_scale"])
    # the shared pages, once: they lie before every tree
    kv = s["kv"].view(torch.uint8)
    rest = kv[s["table"][:, P:].long().clamp(min=0)].view(torch.float8_e4m3fn).float()  # [B, own pages, H, 128, 256]
    own_keys = rest.shape[1] * PAGE
    rest = rest.permute(2, 0, 1, 3, 4).reshape(H, B, own_keys, 2 * D)
    s2 = torch.matmul(q.reshape(H, B, n * G, D), rest[..., :D].transpose(-1, -2))
    # which keys a token sees: all before the tree, and of the tree by its mask's bits
    node = P * PAGE + torch.arange(own_keys, device=dev) - s["first"].long()[:, None]  # [B, keys]
    word = torch.zeros((B, n, s["mask"].shape[1]), dtype=torch.long, device=dev)
    word[b, i] = s["mask"].long() & 0xFFFFFFFF
    at = node.clamp(0, n - 1)
    bit = word.gather(2, (at // 32)[:, None].expand(B, n, -1)) >> (at % 32)[:, None] & 1
    seen = (node < 0)[:, None] | ((node < n)[:, None] & (bit > 0))
    s2 = s2.view(H, B, n, G, own_keys).masked_fill_(~seen[None, :, :, None], -math.inf)
    top = s2.amax(-1)
    if P:
        first = kv[s["table"][0, :P].long()].view(torch.float8_e4m3fn).float().permute(1, 0, 2, 3).reshape(H, P * PAGE, 2 * D)
        s1 = torch.matmul(q.reshape(H, -1, D), first[..., :D].transpose(-1, -2)).view(H, B, n, G, P * PAGE)
        top = torch.maximum(top, s1.amax(-1))
    p2 = s2.sub_(top[..., None]).exp_()
    total = p2.sum(-1)
    out = torch.matmul(p2.view(H, B, n * G, own_keys), rest[..., D:]).view(H, B, n, G, D)
    if P:
        p1 = s1.sub_(top[..., None]).exp_()
        total = total + p1.sum(-1)
        out = out + torch.matmul(p1.view(H, -1, P * PAGE), first[..., D:]).view(H, B, n, G, D)
    out = out / total[..., None] * s["v_scale"]
    lse = top + total.log()
    out = out.permute(1, 2, 0, 3, 4)[b, i].reshape(s["T"], H * G, D)
    return [out.to(torch.bfloat16), lse.permute(1, 2, 0, 3)[b, i].reshape(s["T"], H * G).contiguous()]


def _plain_accept(s):
    B, n = s["case"]["B"], s["max_q"]
    parent, drafts, chosen = (_padded(s, s[k].long(), -1) for k in ("parents", "drafts", "chosen"))
    at = torch.arange(n, device="cuda")
    there = at < s["cu_q"].diff()[:, None]
    child = parent[..., None] == at  # [B, node, its parent]
    match = (there & (parent >= 0) & (drafts == chosen.gather(1, parent.clamp(min=0))))[..., None] & child
    # of the children that the target's token matches, the first alone stands
    first = torch.where(match, at[:, None], n).amin(1)
    stands = (match & (at[:, None] == first[:, None])).any(-1) | (at == 0)
    up = _ancestors(s)
    on = there & (up <= stands[:, None]).all(-1)  # every ancestor stands
    count = on.sum(1)  # with the root
    path = torch.where(on, at, n).sort(1).values
    path = torch.where(path < n, path, -1)
    best = path.clamp(min=0)
    follow = torch.cat((path[:, 1:], torch.full_like(path[:, :1], -1)), 1)
    end = chosen.gather(1, path.gather(1, count[:, None] - 1))
    tokens = torch.where(follow >= 0, drafts.gather(1, follow.clamp(min=0)), torch.where(at == count[:, None] - 1, end, -1))
    # rows of the cache: the path's nodes to the places behind the context
    src = s["first"].long()[:, None] + best
    dst = s["first"].long()[:, None] + at
    move = path >= 0
    rows = torch.arange(B, device="cuda")[:, None].expand(B, n)[move]
    src, dst = src[move], dst[move]
    pages = s["table"].long()[rows, src // PAGE], s["table"].long()[rows, dst // PAGE]
    out = []
    for kv in s["kv"]:
        if s["case"]["fmt"] == "e4m3":
            x = kv.view(torch.uint8)
            x[pages[1], :, dst % PAGE] = x[pages[0], :, src % PAGE]
            out.append(kv)
        else:
            for part, size in ((kv[..., :PAGE * 64], 64), (kv[..., PAGE * 64:], 8)):
                x = part.view(*kv.shape[:3], PAGE, size)
                x[pages[1], :, :, dst % PAGE] = x[pages[0], :, :, src % PAGE]
            out.append(kv)
    return [tokens.to(torch.int32), (count - 1).to(torch.int32), path.to(torch.int32), out]


def _plain_logprobs(s):
    x, T, V = s["logits"].float(), s["case"]["T"], s["case"]["V"]
    at = s["tokens"].long()[:, None]
    top = x.amax(-1, keepdim=True)
    shifted = x - top
    p = shifted.exp()
    total = p.sum(-1, keepdim=True)
    norm = total.log()
    entropy = norm[:, 0] - (p * shifted).sum(-1) / total[:, 0]
    logprob = (shifted.gather(1, at) - norm)[:, 0]
    mine = x.gather(1, at)
    rank = ((x > mine) | ((x == mine) & (torch.arange(V, device="cuda") < at))).sum(-1)
    # values and places as one whole number whose order is that of the value, and of equal ones that of the lower place
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 20) + (V - 1 - torch.arange(V, device="cuda"))
    best = V - 1 - (key.topk(s["case"]["top"], -1).values & ((1 << 20) - 1))
    return [logprob, rank.to(torch.int32), entropy, best.to(torch.int32), shifted.gather(1, best) - norm]


# --------------------------------------------------------------------------- one pass


def run(s):
    op, case = s["op"], s["case"]
    if own:
        import block_sparse_attention_prefill_gb300 as msa

        if op == "rope":
            fp4 = case["fmt"] == "nvfp4"
            write = msa.msa_rope_write_nvfp4 if fp4 else msa.msa_rope_write
            q = write(s["rope"], s["q"], s["k"], s["v"], s["kv"], s["q_scale"], s["k_scale"], s["v_scale"], s["table"], s["cu_q"], s["cu_k"],
                      positions=s["positions"])
            return [q, msa.msa_nvfp4_to_e4m3(s["kv"]) if fp4 else s["kv"]]
        if op == "mask":
            return msa.msa_tree_mask(s["parents"], s["cu_q"], s["cu_k"], s["max_q"])
        if op == "attend":
            return msa.msa_tree_attention(s["q"], s["kv"], s["q_scale"], s["k_scale"], s["v_scale"], s["softmax_scale"], s["table"], s["cu_q"], s["cu_k"],
                                          s["mask"], s["prefix"], s["max_q"], s["max_k"])
        if op == "accept":
            accept = msa.msa_tree_accept_nvfp4 if case["fmt"] == "nvfp4" else msa.msa_tree_accept
            tokens, accepted, path = accept(s["drafts"], s["parents"], s["chosen"], s["cu_q"], s["cu_k"], s["max_q"], kv=s["kv"], block_table=s["table"])
            return [tokens, accepted, path, s["kv"]]
        return msa.msa_logprobs(s["logits"], s["tokens"], top=case["top"])
    return {"rope": _plain_rope, "mask": _plain_mask, "attend": _plain_attend, "accept": _plain_accept, "logprobs": _plain_logprobs}[op](s)


def work(case):
    if case["op"] == "logprobs":
        es = torch.empty((), dtype=TYPES[case["type"]]).element_size()
        return {"bytes": case["T"] * (case["V"] * es + 16 + 8 * case["top"]), "flops": 5 * case["T"] * case["V"]}
    q, seq = _lengths(case)
    T, n = sum(q), max(q)
    if case["op"] == "rope":
        values = T * case["heads"] * 2 * D
        wide = torch.empty((), dtype=TYPES[case["type"]]).element_size()
        queries = T * case["hq"] * D
        bytes_ = (values + queries) * wide + queries * (1 if case["q8"] else 2) + values * (1.0 if case["fmt"] == "e4m3" else 0.5625) + 4 * T * case["axes"]
        if case["fmt"] == "nvfp4":  # the pool is given back as the E4M3 pool that it stands for
            bytes_ += (sum(-(-m // PAGE) for m in seq) + 3) * case["heads"] * (2 * SLOT + PAGE * 2 * D)
        return {"bytes": bytes_, "flops": (queries + values / 2) * 6}
    if case["op"] == "mask":
        return {"bytes": T * (8 + 4 * -(-n // 32)), "flops": T}
    if case["op"] == "attend":
        shared = case["prefix"] * PAGE
        pairs = sum(k * m for k, m in zip(q, seq))  # pairs of a query token and a key, those of the tree with them
        pool = (shared + sum(m - shared for m in seq)) * case["heads"] * 2 * D
        return {"bytes": pool + T * (case["hq"] * (D + 2 * D + 4) + 4 * -(-n // 32)), "flops": 4 * D * case["hq"] * pairs}
    # a path of about five nodes a request, its rows read and written; the tree's words
    row = 2 * D if case["fmt"] == "e4m3" else 144
    moved = sum(min(k - 1, 4) for k in q) * case["layers"] * case["heads"] * row * 2
    return {"bytes": T * 12 + case["B"] * (8 * n + 4) + moved, "flops": T}


# --------------------------------------------------------------------------- the definition in 64 bits


def _value8(code):
    """The real values of E4M3 codes."""
    c = code.long()
    e, m = c >> 3 & 15, c & 7
    x = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8), m * 2.0 ** -9)
    return torch.where(c >= 128, -x, x)


def _exact_turn(case, s, x, weight):
    """Rows turned request by request and pair by pair as complex numbers."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
    y, half = x.clone(), case["rot"] // 2
    pos = s["positions"].reshape(case["axes"], -1).double()
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
        angle = pos[0 if s["axes"] is None else s["axes"][j]] * float(s["inv_freq"][j])
        z = torch.complex(x[..., i0], x[..., i1]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        y[..., i0], y[..., i1] = z.real, z.imag
    return y


def _exact_rope(case, s):
    q = _exact_turn(case, s, s["q"], s["q_norm"])
    if case["q8"]:
        q = (q / s["q_scale"]).clamp(-E4M3_MAX, E4M3_MAX)
    if case["fmt"] == "nvfp4":
        return [q, None]  # what four bits hold is far from what was given
    k, pool = _exact_turn(case, s, s["k"], s["k_norm"]), _value8(s["kv"].view(torch.uint8))
    lens, seq = _lengths(case)
    at = 0
    for b, (n, m) in enumerate(zip(lens, seq)):
        pos = torch.arange(m - n, m, device="cuda")
        page = s["table"][b].long()[pos // PAGE]
        pool[page, :, pos % PAGE, :D] = (k[at:at + n] / s["k_scale"]).clamp(-E4M3_MAX, E4M3_MAX)
        pool[page, :, pos % PAGE, D:] = (s["v"][at:at + n].double() / s["v_scale"]).clamp(-E4M3_MAX, E4M3_MAX)
        at += n
    return [q, pool]


def _exact_attend(case, s):
    lens, seq = _lengths(case)
    G = case["hq"] // case["heads"]
    table, kv, parents = s["table"].cpu().long(), s["kv"].view(torch.uint8), s["parents"].tolist()
    out = torch.empty((s["T"], case["hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["T"], case["hq"]), dtype=torch.float64, device="cuda")
    query = _value8(s["q"].view(torch.uint8)) * s["q_scale"]
    at = 0
    for b, (n, m) in enumerate(zip(lens, seq)):
        seen = torch.zeros((n, m), dtype=torch.bool)
        seen[:, :m - n] = True
        for i in range(n):
            j = i
            while j >= 0:  # a token's way up to the root
                seen[i, m - n + j] = True
                j = parents[at + j]
        seen = seen.cuda().repeat_interleave(G, 0)
        pages = table[b, :-(-m // PAGE)].cuda()
        for h in range(case["heads"]):
            x = _value8(kv[pages, h]).reshape(-1, 2 * D)[:m]
            z = query[at:at + n, h * G:(h + 1) * G].reshape(-1, D) @ x[:, :D].T * (s["k_scale"] * s["softmax_scale"])
            z.masked_fill_(~seen, -math.inf)
            lse[at:at + n, h * G:(h + 1) * G] = torch.logsumexp(z, -1).view(n, G)
            out[at:at + n, h * G:(h + 1) * G] = (torch.softmax(z, -1) @ x[:, D:] * s["v_scale"]).view(n, G, D)
        at += n
    return [out, lse]


def _exact_logprobs(case, s):
    logprob, entropy, top = [], [], []
    step = max(1, (1 << 26) // case["V"])
    for a in range(0, case["T"], step):
        z = torch.log_softmax(s["logits"][a:a + step].double(), -1)
        logprob.append(z.gather(1, s["tokens"][a:a + step].long()[:, None])[:, 0])
        entropy.append(-(z.exp() * z).sum(-1))
        top.append(z.sort(-1, descending=True).values[:, :case["top"]])
    return [torch.cat(logprob), None, torch.cat(entropy), None, torch.cat(top)]


def exact(case, seed):
    if case["op"] in ("mask", "accept"):
        return None  # whole numbers, and rows moved as they are
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](case, s)
