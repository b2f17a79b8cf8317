"""The cache and verification operators around block-sparse attention: cases, plain forms and exact results.

Five operators that a server calls next to ``msa_plan`` / ``msa_prefill`` / ``msa_decode``:

  write    new K/V tokens are quantised and written into their pages (E4M3 or NVFP4)
  read     tokens of the paged cache are read back, dequantised, as contiguous K and V
  attend   dense causal attention of a batch whose requests share their first pages: the shared pages' part is computed once for all
  verify   drafted tokens are accepted or replaced against the target's probabilities from given random numbers
  greedy   drafted tokens are accepted while they are the target's best token

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
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one step of speculative decoding: 64 requests append 8 tokens each (latency)
        {"name": "write decode 64x8", "op": "write", "fmt": "e4m3", "type": "bf16", "heads": 2, "B": 64, "q_lo": 8, "q_hi": 8, "ctx": 4096, "lens": 1},
        # a large prefill batch: 8 chunks of about 8k tokens, 8 KV heads (bandwidth)
        {"name": "write prefill 8 x 8k", "op": "write", "fmt": "e4m3", "type": "bf16", "heads": 8, "B": 8, "q_lo": 7001, "q_hi": 8192, "ctx": 9000, "lens": 2},
        # ragged chunked prefill into NVFP4 pages, and the chunk read back as the attention sees it
        {"name": "write nvfp4 and read back", "op": "write", "fmt": "nvfp4", "type": "fp16", "heads": 2, "B": 8, "q_lo": 128, "q_hi": 4096, "ctx": 32768, "lens": 3},
        # a whole 1M-token context read back in bf16
        {"name": "read 1M tokens", "op": "read", "fmt": "e4m3", "type": "bf16", "heads": 2, "B": 1, "q_lo": 1048576, "q_hi": 1048576, "ctx": 1048576, "lens": 4},
        # parts of 16 NVFP4 requests from odd positions, in fp32
        {"name": "read nvfp4 16 parts", "op": "read", "fmt": "nvfp4", "type": "fp32", "heads": 2, "B": 16, "q_lo": 300, "q_hi": 9001, "ctx": 32768, "lens": 5},
        # plain decode of 16 requests behind one 32k-token system prompt
        {"name": "attend 16x1 over 32k", "op": "attend", "hq": 16, "heads": 2, "B": 16, "q_lo": 1, "q_hi": 1, "prefix": 256, "own_lo": 1, "own_hi": 500, "lens": 6},
        # speculative verify of 64 requests behind a 128k-token shared document
        {"name": "attend 64x8 over 128k", "op": "attend", "hq": 16, "heads": 2, "B": 64, "q_lo": 8, "q_hi": 8, "prefix": 1024, "own_lo": 8, "own_hi": 2000, "lens": 7},
        # nothing shared: 16 requests of up to 128k tokens of their own
        {"name": "attend 16x8 own 128k", "op": "attend", "hq": 16, "heads": 2, "B": 16, "q_lo": 8, "q_hi": 8, "prefix": 0, "own_lo": 32768, "own_hi": 131072, "lens": 8},
        # ragged chunks of new prompts behind an 8k-token shared prefix, groups of 3 query heads
        {"name": "attend 5 chunks over 8k", "op": "attend", "hq": 12, "heads": 4, "B": 5, "q_lo": 1, "q_hi": 700, "prefix": 65, "own_lo": 700, "own_hi": 1500, "lens": 9},
        # one request, three drafts, a small vocabulary (latency)
        {"name": "verify 1x3 of 32k", "op": "verify", "type": "fp32", "B": 1, "k": 3, "V": 32000},
        # 64 requests, seven drafts, a large odd vocabulary
        {"name": "verify 64x7 of 200k", "op": "verify", "type": "fp32", "B": 64, "k": 7, "V": 200003},
        # the same step decided greedily on bf16 logits
        {"name": "greedy 64x7 of 131k", "op": "greedy", "type": "bf16", "B": 64, "k": 7, "V": 131072},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "verify", "greedy"))
    lens = rng.randrange(1, 1 << 20)
    if op in ("write", "read"):
        heads, B = rng.choice((1, 2, 3, 4, 8)), _log(rng, 1, 64)
        most = max(1, 131072 // (B * heads))  # tokens a request: B * heads * most is at most the largest write's
        hi = _log(rng, 1, most)
        return {"op": op, "fmt": rng.choice(("e4m3", "nvfp4")), "type": rng.choice(tuple(TYPES)), "heads": heads, "B": B,
                "q_lo": rng.randint(1, hi), "q_hi": hi, "ctx": hi + _log(rng, 1, 4096), "lens": lens}
    if op == "attend":
        heads, group = rng.choice(((1, 1), (1, 16), (2, 4), (2, 8), (4, 3), (8, 4)))
        hi = rng.choice((1, 1, 2, 4, 8, _log(rng, 9, 400)))
        B = _log(rng, 1, max(1, min(64, 8192 // (heads * group * hi))))
        most = max(2, min(1024, 2 ** 23 // (B * heads * group * hi)))  # pages: rows x keys below the largest case's
        prefix = rng.choice((0, _log(rng, 1, most), _log(rng, 1, most)))
        own_hi = hi + _log(rng, 1, PAGE * (min(most, 64) if prefix else most))
        return {"op": op, "hq": heads * group, "heads": heads, "B": B, "q_lo": rng.randint(1, hi), "q_hi": hi, "prefix": prefix,
                "own_lo": rng.randint(hi, own_hi), "own_hi": own_hi, "lens": lens}
    return {"op": op, "type": rng.choice(tuple(TYPES)), "B": _log(rng, 1, 64), "k": rng.choice((0, 1, 2, 3, 4, 5, 6, 7)), "V": _log(rng, 500, 200003)}


# --------------------------------------------------------------------------- inputs


def _lengths(case):
    """Per request: how many tokens the call handles, and the request's length (they are its last tokens, or start at an odd place when read)."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    if case["op"] == "attend":
        q[0] = case["q_hi"]
        seq = [case["prefix"] * PAGE + max(n, r.randint(case["own_lo"], case["own_hi"])) for n in q]
    else:
        seq = [r.randint(n, max(n, case["ctx"])) for n in q]
    return q, seq


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
    own_pages = [p - shared for p in pages]
    total = shared + sum(own_pages) + spare
    perm = torch.from_numpy(np.random.RandomState(r).permutation(total).astype("int32"))
    table = torch.full((len(seq), max(max(pages), 1)), -1, dtype=torch.int32)
    at = shared
    for b, p in enumerate(own_pages):
        table[b, :shared] = perm[:shared]
        table[b, shared:shared + p] = perm[at:at + p]
        at += p
    return table.to(dev), total


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] in ("write", "read"):
        q, seq = _lengths(case)
        s["table"], pages = _table(seq, 0, 3, seed % (1 << 31), dev)
        s["cu_q"], s["cu_k"], s["T"] = _cum(q, dev), _cum(seq, dev), sum(q)
        s["dtype"] = TYPES[case["type"]]
        s["start"] = torch.tensor([a - n for a, n in zip(seq, q)], dtype=torch.int32, device=dev)
        make = _pool4 if case["fmt"] == "nvfp4" else _pool
        s["kv"], scale = make(pages, case["heads"], g, dev)
        if case["op"] == "write":
            # K and V as a fused projection leaves them: parts of one row a token, behind the query's part
            x = _normal((s["T"], 4, case["heads"], D), g, dev).to(s["dtype"])
            s["k"], s["v"] = x[:, 2], x[:, 3]
        s["k_scale"], s["v_scale"] = scale, _float32(scale * 1.2345)
        return s
    if case["op"] == "attend":
        q, seq = _lengths(case)
        s["table"], pages = _table(seq, case["prefix"], 2, seed % (1 << 31), dev)
        s["cu_q"], s["cu_k"], s["T"] = _cum(q, dev), _cum(seq, dev), sum(q)
        s["kv"], s["k_scale"] = _pool(pages, case["heads"], g, dev)
        s["v_scale"] = s["k_scale"]
        s["q_scale"] = _float32(5.7139 / E4M3_MAX)
        x = _normal((s["T"], case["hq"], D), g, dev)
        s["q"] = (x / s["q_scale"]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["softmax_scale"] = 1.0 / math.sqrt(D)
        s["max_q"], s["max_k"], s["prefix"] = max(q), max(seq), case["prefix"]
        return s
    B, k, V, t = case["B"], case["k"], case["V"], TYPES[case["type"]]
    if case["op"] == "verify":
        # peaked distributions, as language models give them; the draft model's are near the target's
        z = _normal((B, k + 1, V), g, dev)
        y = _normal((B, k, V), g, dev)
        target, draft = torch.softmax(3 * z, -1), torch.softmax(3 * z[:, :k] + 0.8 * y, -1)
        cut = draft.reshape(B * k, V).double().cumsum(-1)
        u = torch.rand((B * k, 1), generator=g, device=dev, dtype=torch.float64) * cut[:, -1:]
        s["drafts"] = torch.searchsorted(cut, u).clamp_(max=V - 1).reshape(B, k).to(torch.int32)  # sampled from the draft
        s["target"], s["draft"] = target.to(t), draft.to(t)
        s["u"] = torch.rand((B, k + 1), generator=g, device=dev)
    else:
        s["target"] = (3 * _normal((B, k + 1, V), g, dev)).to(t)
        best = s["target"][:, :k].float().argmax(-1).to(torch.int32)
        miss = torch.rand((B, k), generator=g, device=dev) < 0.3
        other = torch.randint(0, V, (B, k), generator=g, device=dev, dtype=torch.int32)
        s["drafts"] = torch.where(miss, other, best)
    # some requests had fewer drafts than the batch's most
    s["count"] = torch.randint(max(0, k - 2), k + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    return s


# --------------------------------------------------------------------------- plain forms


def _places(s):
    """(request, position, page, row in the page) of every token that the call handles."""
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    pos = s["start"].long()[b] + t - s["cu_q"].long()[b]
    return b, pos, s["table"].long()[b, pos // PAGE], pos % PAGE


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
    """Codes [..., 64] and E4M3 scales [..., 8] -> what the attention reads: E4M3(code x scale), as fp32 [..., 128]."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = grid[torch.stack((codes & 15, codes >> 4), -1).long()].reshape(*codes.shape[:-1], 8, 16) * scales.float().unsqueeze(-1)
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float().reshape(*codes.shape[:-1], D)


def _plain_write(s):
    _, _, page, row = _places(s)
    kv = s["kv"]
    for half, x, g in ((0, s["k"], s["k_scale"]), (1, s["v"], s["v_scale"])):
        if s["case"]["fmt"] == "e4m3":
            code = (x.float() / g).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            kv.view(torch.uint8)[page, :, row, half * D:(half + 1) * D] = code.view(torch.uint8)
        else:
            codes, scale = _encode4(x.float(), g)
            kv[:, :, half, :PAGE * 64].view(*kv.shape[:2], PAGE, 64)[page, :, row] = codes
            kv[:, :, half, PAGE * 64:].view(*kv.shape[:2], PAGE, 8)[page, :, row] = scale.view(torch.uint8)


def _plain_read(s):
    _, _, page, row = _places(s)
    kv, out = s["kv"], []
    for half, g in ((0, s["k_scale"]), (1, s["v_scale"])):
        if s["case"]["fmt"] == "e4m3":
            x = kv.view(torch.uint8)[page, :, row, half * D:(half + 1) * D].view(torch.float8_e4m3fn).float()
        else:
            x = _decode4(kv[:, :, half, :PAGE * 64].view(*kv.shape[:2], PAGE, 64)[page, :, row],
                         kv[:, :, half, PAGE * 64:].view(*kv.shape[:2], PAGE, 8)[page, :, row].view(torch.float8_e4m3fn))
        out.append((x * g).to(s["dtype"]))
    return out


def _plain_attend(s):
    case, P = s["case"], s["prefix"]
    B, H, G, n = case["B"], case["heads"], case["hq"] // case["heads"], s["max_q"]
    dev = s["q"].device
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    q_len, seq = cu_q.diff(), cu_k.diff()
    t = torch.arange(s["T"], device=dev)
    b = torch.searchsorted(cu_q[1:], t, right=True)
    i = t - cu_q[b]
    # queries padded to the longest chunk, [H, B, n, G, D]; their positions
    q = torch.zeros((B, n, H, G, D), device=dev)
    q[b, i] = s["q"].float().view(-1, H, G, D)
    q = q.permute(2, 0, 1, 3, 4) * (s["q_scale"] * s["k_scale"] * s["softmax_scale"])
    pos = (seq - q_len)[:, None] + torch.arange(n, device=dev)
    # the shared pages, once: they lie before every query
    kv = s["kv"].view(torch.uint8)
    rest = kv[s["table"][:, P:].long().clamp(min=0)].view(torch.float8_e4m3fn).float()  # [B, own pages, H, 128, 256]
    own_keys = rest.shape[1] * PAGE
    rest = rest.permute(2, 0, 1, 3, 4).reshape(H, B, own_keys, 2 * D)
    s2 = torch.matmul(q.reshape(H, B, n * G, D), rest[..., :D].transpose(-1, -2))
    key = P * PAGE + torch.arange(own_keys, device=dev)
    s2 = s2.view(H, B, n, G, own_keys).masked_fill_((key > pos[..., None])[None, :, :, None], -math.inf)
    top = s2.amax(-1)
    if P:
        first = kv[s["table"][0, :P].long()].view(torch.float8_e4m3fn).float().permute(1, 0, 2, 3).reshape(H, P * PAGE, 2 * D)
        s1 = torch.matmul(q.reshape(H, -1, D), first[..., :D].transpose(-1, -2)).view(H, B, n, G, P * PAGE)
        top = torch.maximum(top, s1.amax(-1))
    p2 = s2.sub_(top[..., None]).exp_()
    total = p2.sum(-1)
    # keys past a request's end have probability 0; what their values are does not matter
    out = torch.matmul(p2.view(H, B, n * G, own_keys), rest[..., D:]).view(H, B, n, G, D)
    if P:
        p1 = s1.sub_(top[..., None]).exp_()
        total = total + p1.sum(-1)
        out = out + torch.matmul(p1.view(H, -1, P * PAGE), first[..., D:]).view(H, B, n, G, D)
    out = out / total[..., None] * s["v_scale"]
    lse = top + total.log()
    out = out.permute(1, 2, 0, 3, 4)[b, i].reshape(s["T"], H * G, D)
    return [out.to(torch.bfloat16), lse.permute(1, 2, 0, 3)[b, i].reshape(s["T"], H * G).contiguous()]


def _answer(s, accepted, token):
    B, n = s["target"].shape[:2]
    at = torch.arange(n, device="cuda")
    drafts = torch.nn.functional.pad(s["drafts"], (0, 1), value=-1)
    tokens = torch.where(at < accepted[:, None], drafts, torch.where(at == accepted[:, None], token[:, None].to(torch.int32), torch.full_like(drafts, -1)))
    return [tokens, accepted.to(torch.int32)]


def _plain_verify(s):
    target, draft, u = s["target"], s["draft"], s["u"]
    B, n, V = target.shape
    k = n - 1
    rows = torch.arange(B, device="cuda")
    at = s["drafts"].long()[..., None]
    p, q = target[:, :k].gather(2, at)[..., 0].double(), draft.gather(2, at)[..., 0].double()
    ok = (u[:, :k].double() * q < p) & (torch.arange(k, device="cuda") < s["count"][:, None])  # exact in 64 bits
    accepted = ok.long().cumprod(1).sum(1)
    w = target[rows, accepted].float()
    if k:
        w = w - torch.where((accepted < s["count"])[:, None], draft[rows, accepted.clamp(max=k - 1)].float(), torch.zeros((), device="cuda"))
    # weights in steps of 2^-44, so that their sums are exact and no order of adding matters
    w = (w.clamp(0, 1) * 2.0 ** 44).long()
    cut = w.cumsum(1)
    total = cut[:, -1]
    x = (u[:, -1].double() * 2 ** 31).long().clamp(0, 2 ** 31 - 1)
    t = x * (total >> 31) + (x * (total & (2 ** 31 - 1)) >> 31)  # floor(u * total)
    return _answer(s, accepted, (cut <= t[:, None]).sum(1))


def _first_best(x):
    """The lowest index of the largest value of each row."""
    top = x.amax(-1, keepdim=True)
    V = x.shape[-1]
    return torch.where(x == top, torch.arange(V, device=x.device), V).amin(-1)


def _plain_greedy(s):
    k = s["target"].shape[1] - 1
    best = _first_best(s["target"].float())
    ok = (best[:, :k] == s["drafts"]) & (torch.arange(k, device="cuda") < s["count"][:, None])
    accepted = ok.long().cumprod(1).sum(1)
    return _answer(s, accepted, best.gather(1, accepted[:, None])[:, 0])


# --------------------------------------------------------------------------- one pass


def run(s):
    op, case = s["op"], s["case"]
    if own:
        import block_sparse_attention_prefill_gb300 as msa

        if op in ("write", "read"):
            fp4 = case["fmt"] == "nvfp4"
            if op == "write":
                write = msa.msa_kv_write_nvfp4 if fp4 else msa.msa_kv_write
                write(s["k"], s["v"], s["kv"], s["k_scale"], s["v_scale"], s["table"], s["cu_q"], s["cu_k"])
                if not fp4:
                    return s["kv"]
            read = msa.msa_kv_read_nvfp4 if fp4 else msa.msa_kv_read
            return read(s["kv"], s["k_scale"], s["v_scale"], s["table"], s["cu_q"], s["T"], starts=s["start"], dtype=s["dtype"])
        if op == "attend":
            return msa.msa_prefix_attention(s["q"], s["kv"], s["q_scale"], s["k_scale"], s["v_scale"], s["softmax_scale"], s["table"], s["cu_q"], s["cu_k"],
                                            s["prefix"], s["max_q"], s["max_k"])
        if op == "verify":
            return msa.msa_verify(s["target"], s["drafts"], s["u"], draft_probs=s["draft"], num_drafts=s["count"])
        return msa.msa_verify_greedy(s["target"], s["drafts"], num_drafts=s["count"])
    if op == "write":
        _plain_write(s)
        return s["kv"] if case["fmt"] == "e4m3" else _plain_read(s)
    return {"read": _plain_read, "attend": _plain_attend, "verify": _plain_verify, "greedy": _plain_greedy}[op](s)


def work(case):
    if case["op"] in ("write", "read"):
        values = sum(_lengths(case)[0]) * case["heads"] * 2 * D
        wide = values * torch.empty((), dtype=TYPES[case["type"]]).element_size()
        packed = values * (1.0 if case["fmt"] == "e4m3" else 0.5625)
        back = case["op"] == "write" and case["fmt"] == "nvfp4"  # the cache read and the tokens written once more
        return {"bytes": (wide + packed) * (2 if back else 1), "flops": 2 * values}
    if case["op"] == "attend":
        q, seq = _lengths(case)
        shared = case["prefix"] * PAGE
        keys = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, seq))  # pairs of a query token and a key
        pool = (shared + sum(m - shared for m in seq)) * case["heads"] * 2 * D
        return {"bytes": pool + sum(q) * case["hq"] * (D + 2 * D + 4), "flops": 4 * D * case["hq"] * keys}
    es = torch.empty((), dtype=TYPES[case["type"]]).element_size()
    if case["op"] == "greedy":
        return {"bytes": case["B"] * (case["k"] + 1) * case["V"] * es, "flops": case["B"] * (case["k"] + 1) * case["V"]}
    # one row of the target a request, and the draft's where a draft was refused
    return {"bytes": case["B"] * case["V"] * es * (2 if case["k"] else 1), "flops": 3 * case["B"] * case["V"]}


# --------------------------------------------------------------------------- the definition in 64 bits


def _round_to(x, mantissa, least, most):
    """float64 values rounded, ties to even, to a format of `mantissa` fraction bits with its smallest normal exponent `least` and largest value `most`."""
    e = torch.frexp(x.abs())[1].double() - 1
    step = torch.exp2(e.clamp(min=least) - mantissa)
    return (torch.round(x / step) * step).clamp(-most, most)


def _rows_of(case, s):
    """[T] page and row of the tokens that a call handles, found request by request."""
    q, seq = _lengths(case)
    page, row = [], []
    table = s["table"].cpu()
    for b, (n, m) in enumerate(zip(q, seq)):
        pos = torch.arange(m - n, m)
        page.append(table[b].long()[pos // PAGE])
        row.append(pos % PAGE)
    return torch.cat(page).cuda(), torch.cat(row).cuda()


def _value8(code):
    """The real values of E4M3 codes."""
    c = code.long()
    e, m = c >> 3 & 15, c & 7
    x = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8), m * 2.0 ** -9)
    return torch.where(c >= 128, -x, x)


def _exact_write(case, s):
    page, row = _rows_of(case, s)
    if case["fmt"] == "e4m3":
        pool = _value8(s["kv"].view(torch.uint8))
        for half, x, g in ((0, s["k"], s["k_scale"]), (1, s["v"], s["v_scale"])):
            pool[page, :, row, half * D:(half + 1) * D] = _round_to(x.double() / g, 3, -6, E4M3_MAX)
        return pool
    out = []
    for x, g in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x = x.double().reshape(*x.shape[:-1], 8, 16)
        scale = _round_to(x.abs().amax(-1, keepdim=True) / (6 * g), 3, -6, E4M3_MAX)
        code = _round_to(torch.where(scale > 0, x / (scale * g), torch.zeros_like(x)), 1, 0, E2M1_MAX)
        out.append((_round_to(code * scale, 3, -6, E4M3_MAX) * g).reshape(*x.shape[:-2], D))
    return out


def _exact_read(case, s):
    page, row = _rows_of(case, s)
    kv, out = s["kv"].view(torch.uint8), []
    for half, g in ((0, s["k_scale"]), (1, s["v_scale"])):
        if case["fmt"] == "e4m3":
            x = _value8(kv[page, :, row, half * D:(half + 1) * D])
        else:
            slot = kv[:, :, half]
            codes = slot[..., :PAGE * 64].reshape(*slot.shape[:2], PAGE, 64)[page, :, row].long()
            scale = _value8(slot[..., PAGE * 64:].reshape(*slot.shape[:2], PAGE, 8)[page, :, row])
            nibble = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
            e, m = nibble // 2 % 4, nibble % 2
            x = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m / 2), m / 2)
            x = torch.where(nibble >= 8, -x, x) * scale.repeat_interleave(16, -1)
            x = _round_to(x, 3, -6, E4M3_MAX)
        out.append(x * g)
    return out


def _exact_attend(case, s):
    q_lens, seq = _lengths(case)
    G = case["hq"] // case["heads"]
    table, kv = s["table"].cpu().long(), s["kv"].view(torch.uint8)
    out = torch.empty((s["T"], case["hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["T"], case["hq"]), dtype=torch.float64, device="cuda")
    query = _value8(s["q"].view(torch.uint8)) * s["q_scale"]
    at = 0
    for b, (n, m) in enumerate(zip(q_lens, seq)):
        pages = table[b, :-(-m // PAGE)].cuda()
        for h in range(case["heads"]):
            x = _value8(kv[pages, h]).reshape(-1, 2 * D)[:m]
            z = query[at:at + n, h * G:(h + 1) * G].reshape(-1, D) @ x[:, :D].T * (s["k_scale"] * s["softmax_scale"])
            i = torch.arange(m - n, m, device="cuda").repeat_interleave(G)
            z.masked_fill_(torch.arange(m, device="cuda") > i[:, None], -math.inf)
            lse[at:at + n, h * G:(h + 1) * G] = torch.logsumexp(z, -1).view(n, G)
            out[at:at + n, h * G:(h + 1) * G] = (torch.softmax(z, -1) @ x[:, D:] * s["v_scale"]).view(n, G, D)
        at += n
    return [out, lse]


def exact(case, seed):
    if case["op"] in ("verify", "greedy"):
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)
