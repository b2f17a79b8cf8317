"""Trees of drafted tokens: masks, attention and acceptance against plain
implementations (the attention in 64 bits, with the tolerance that
test_prefix_attention_gpu derives; masks, tokens and moved rows equal)."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_prefix_attention_gpu import KS, QS, SM, VS, _batch

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
cum = lambda v: i32(np.concatenate([[0], np.cumsum(v)]).astype(int).tolist())  # noqa: E731


def _parents(n, kind, r):
    if not n:
        return []
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "two":  # two chains in turn
        return [-1] + [max(0, i - 2) for i in range(1, n)]
    if kind == "forest":
        return [-1 if r.rand() < 0.3 else int(r.randint(i)) if i else -1 for i in range(n)]
    return [-1] + [int(r.randint(max(0, i - 9), i)) for i in range(1, n)]


def _seen(parents):
    n = len(parents)
    m = np.eye(n, dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] |= m[p]
    return m


def _words(m, width):
    out = np.zeros((m.shape[0], width), np.uint32)
    for i, j in zip(*np.nonzero(m)):
        out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


@pytest.mark.parametrize("kind", ["chain", "star", "two", "forest", "random"])
@pytest.mark.parametrize("lens", [[1], [256], [0, 3, 0, 1], [33, 64, 65, 31, 32], [255, 7, 129]])
def test_mask(lens, kind):
    r = np.random.RandomState(len(lens))
    seqs = [n + int(r.randint(0, 5000)) for n in lens]
    seqs[0] = lens[0]
    parents = [_parents(n, kind, r) for n in lens]
    flat = sum(parents, [])
    most = max(lens)
    W = -(-most // 32)
    pad = 3
    mask, pos = torch.full((len(flat) + pad, W), 77, dtype=torch.int32, device="cuda"), torch.full((len(flat) + pad,), 77, dtype=torch.int32, device="cuda")
    status = i32([0])
    got = msa.msa_tree_mask(i32(flat + [5] * pad), cum(lens), cum(seqs), most, mask=mask, positions=pos, status=status)
    assert got[0] is mask and got[1] is pos and status.item() == 0
    want = np.concatenate([_words(_seen(p), W) for p in parents if p])
    assert np.array_equal(mask[:len(flat)].cpu().numpy(), want) and (mask[len(flat):] == 77).all()
    depth = [s - n + int(d) - 1 for p, n, s in zip(parents, lens, seqs) for d in _seen(p).sum(1)]
    assert pos[:len(flat)].tolist() == depth and (pos[len(flat):] == 77).all()
    new = msa.msa_tree_mask(i32(flat), cum(lens), cum(seqs), most)
    assert torch.equal(new[0], mask[:len(flat)]) and torch.equal(new[1], pos[:len(flat)])


def test_mask_of_bad_parents_and_lengths():
    status = i32([0])
    mask, pos = torch.zeros((6, 1), dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    # a parent that is the node itself, one behind it, one below -1: roots
    msa.msa_tree_mask(i32([-1, 1, 5, -7, 3, 4]), i32([0, 6]), i32([0, 10]), 6, mask=mask, positions=pos, status=status)
    assert status.item() == msa.STATUS_BAD_TREE
    assert mask[:, 0].tolist() == [1, 2, 4, 8, 24, 56] and pos.tolist() == [4, 4, 4, 4, 5, 6]
    # more tokens than the limit, or than the sequence: nothing is written
    for cu_q, cu_k, most in (([0, 2, 6], [0, 2, 8], 3), ([0, 2, 6], [0, 2, 5], 6), ([0, 2, 9], [0, 2, 20], 8), ([-1, 2, 6], [0, 9, 20], 8)):
        status.zero_(), mask.fill_(9), pos.fill_(9)
        msa.msa_tree_mask(i32([-1, 0, -1, 0, 1, 2]), i32(cu_q), i32(cu_k), most, mask=mask, positions=pos, status=status)
        assert status.item() == msa.STATUS_BAD_SEQLENS
        assert (mask[2:] == 9).all() if cu_q[0] == 0 else (mask[:2] == 9).all()


# ------------------------------------------------------------------ attention


def _reference(w, masks, left_out=()):
    hq, hkv = w["q"].shape[1], w["kv"].shape[1]
    G = hq // hkv
    outs, at = [], 0
    table = w["table"].long()
    q = w["q"].double() * (QS * KS * SM)
    for b, (n, m) in enumerate(zip(w["q_lens"], w["seqs"])):
        if not n:
            continue
        pages = table[b, :-(-m // 128)]
        there = torch.tensor([int(x) not in left_out and 0 <= int(x) < w["kv"].shape[0] for x in pages], device="cuda").repeat_interleave(128)[:m]
        x = w["kv"][pages.clamp(0, w["kv"].shape[0] - 1)].double().transpose(0, 1).reshape(hkv, -1, 256)[:, :m].repeat_interleave(G, 0)
        seen = torch.ones((n, m), dtype=torch.bool, device="cuda")
        seen[:, m - n:] = torch.from_numpy(masks[b]).cuda()
        seen &= there
        o = torch.zeros((n, hq, 128), dtype=torch.float64, device="cuda")
        a, lse = o.clone(), torch.full((n, hq), -torch.inf, dtype=torch.float64, device="cuda")
        for i in range(n):  # only the keys that a row sees
            k = seen[i].nonzero()[:, 0]
            if len(k):
                z = torch.einsum("hd,hkd->hk", q[at + i], x[:, k, :128])
                lse[i] = torch.logsumexp(z, -1)
                p = torch.exp(z - lse[i][:, None])
                v = x[:, k, 128:]
                o[i], a[i] = torch.einsum("hk,hkd->hd", p, v), torch.einsum("hk,hkd->hd", p, v.abs())
        outs.append((o * VS, a * VS, lse))
        at += n
    return [torch.cat(x) for x in zip(*outs)]


def _run(w, mask, **kw):
    status = i32([0])
    out, lse = msa.msa_tree_attention(w["q"], w["kv"], QS, KS, VS, SM, w["table"], w["cu_q"], w["cu_k"], mask, w["prefix"], w["max_q"], w["max_k"],
                                      status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, status.item()


def _compare(w, masks, got, left_out=()):
    out, lse = got[0].double(), got[1].double()
    ref, a, ref_lse = _reference(w, masks, left_out)
    assert torch.equal(torch.isnan(out), torch.isnan(ref)) and torch.equal(torch.isnan(lse), torch.isnan(ref_lse))
    err = (out - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -10 * a)
    assert not (err > 0).any(), (err.nan_to_num(-1).max().item(), err.nan_to_num(-1).argmax().item())
    inf = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), inf) and (out[inf] == 0).all()
    ok = ~inf & ~torch.isnan(ref_lse)
    assert ((lse - ref_lse).abs()[ok] <= 2.0 ** -12 + 2.0 ** -20 * ref_lse.abs()[ok]).all()


CASES = [
    # hq, hkv, q_lens, own keys, prefix pages
    (8, 1, [1], [1], 0),
    (8, 1, [1], [129], 3),
    (16, 2, [16] * 3, [16, 100, 1000], 0),
    (16, 2, [64, 33, 1, 50], [64, 160, 128, 700], 5),
    (16, 2, [40, 64], [40, 150], 200),
    (6, 2, [256, 255, 7], [256, 500, 130], 0),
    (4, 4, [200, 3], [210, 90], 1),
    (128, 1, [5, 70], [60, 300], 0),
    (5, 1, [97, 0, 130], [97, 0, 4000], 0),
    (16, 16, [32], [3000], 0),
]


@pytest.mark.parametrize("kind", ["random", "chain", "bits", "few"])
@pytest.mark.parametrize("case", CASES)
def test_attention(case, kind):
    """Trees, and any bits: some rows see nothing of the tree, where no context lies before it nothing at all."""
    hq, hkv, q_lens, own, prefix = case
    w = _batch(hq, hkv, q_lens, own, prefix)
    r = np.random.RandomState(7)
    width = -(-max(q_lens) // 32) + 2
    masks = []
    for n in q_lens:
        masks.append(r.rand(n, n) < (0.5 if kind == "bits" else 0.01) if kind in ("bits", "few") else _seen(_parents(n, kind, r)))
    words = np.concatenate([_words(m, width) for m in masks if m.size])
    # bits behind a request's tokens have no effect
    at = 0
    for n in q_lens:
        for j in range(n, 32 * width):
            if r.rand() < 0.5:
                words.view(np.uint32)[at:at + n, j // 32] |= np.uint32(1 << (j % 32))
        at += n
    got = _run(w, torch.from_numpy(words).cuda())
    assert got[2] == 0
    _compare(w, masks, got)


def test_a_chain_is_causal():
    w = _batch(16, 2, [64, 20, 33], [700, 20, 300], 2)
    mask = torch.from_numpy(np.concatenate([_words(_seen(_parents(n, "chain", None)), 2) for n in (64, 20, 33)])).cuda()
    out, lse, _ = _run(w, mask)
    ref, ref_lse = msa.msa_prefix_attention(w["q"], w["kv"], QS, KS, VS, SM, w["table"], w["cu_q"], w["cu_k"], 2, w["max_q"], w["max_k"])
    # both within their rounding of the same values
    assert ((out.double() - ref.double()).abs() <= 2.0 ** -7 * ref.double().abs() + 2.0 ** -9).all()
    assert ((lse - ref_lse).abs() <= 2.0 ** -11 + 2.0 ** -19 * ref_lse.abs()).all()


def test_nan_is_seen_only_where_the_mask_lets_it():
    """NaN among K and V codes of tree keys reaches the rows that see them, those behind the end or of the context as ever."""
    w = _batch(16, 2, [70, 40], [150, 90], 1)
    r = np.random.RandomState(3)
    masks = [_seen(_parents(n, "random", r)) for n in (70, 40)]
    kv = w["kv"].view(torch.uint8)

    def spot(b, key):
        key += 128
        return int(w["table"][b, key // 128]), key % 128

    p, k = spot(0, 80 + 13)  # node 13 of the first tree: K of head 0, V of head 1
    kv[p, 0, k, 5] = 0x7F
    kv[p, 1, k, 128 + 77] = 0xFF
    p, k = spot(0, 80 + 60)
    kv[p, 0, k, 128 + 3] = 0x7F
    p, k = spot(1, 20)  # context of the second: V
    kv[p, 1, k, 128 + 100] = 0x7F
    p, k = spot(1, 95)  # behind the second's end
    kv[p, :, k] = 0x7F
    got = _run(w, torch.from_numpy(np.concatenate([_words(m, 3) for m in masks])).cuda())
    assert torch.isnan(got[0]).any() and not torch.isnan(got[0]).all()
    _compare(w, masks, got)


def test_bad_pages_and_lengths():
    w = _batch(16, 2, [10, 20], [600, 400], 0)
    masks = [_seen(_parents(n, "chain", None)) for n in (10, 20)]
    mask = torch.from_numpy(np.concatenate([_words(m, 1) for m in masks])).cuda()
    w["table"][0, 1] = 10 ** 6
    w["table"][1, 3] = -5  # the tree's own page: only keys on other pages are left
    got = _run(w, mask)
    assert got[2] == msa.STATUS_BAD_BLOCK
    _compare(w, masks, got, left_out=(10 ** 6, -5))
    w = _batch(16, 2, [10, 20], [600, 400], 0)
    w["max_q"] = 19
    out, lse, status = _run(w, mask)
    assert status == msa.STATUS_BAD_SEQLENS and (out == 0).all() and torch.isneginf(lse).all()


def test_many_requests_and_other_ways_to_call():
    """More requests than one CTA plans for; padding; a graph; another stream; given outputs and workspace."""
    lens = [1 + (7 * i) % 5 for i in range(600)]
    w = _batch(8, 2, lens, [n + (13 * i) % 200 for i, n in enumerate(lens)], 1)
    r = np.random.RandomState(3)
    masks = [_seen(_parents(n, "random", r)) for n in lens]
    mask = torch.from_numpy(np.concatenate([_words(m, 1) for m in masks])).cuda()
    got = _run(w, mask)
    assert got[2] == 0
    _compare(w, masks, got)
    T = sum(lens)
    w["q"] = torch.cat([w["q"].view(torch.uint8), torch.full((9, 8, 128), 0x7F, dtype=torch.uint8, device="cuda")]).view(torch.float8_e4m3fn)
    mask = torch.cat([mask, torch.full((9, 1), -1, dtype=torch.int32, device="cuda")])
    out, lse = torch.full((T + 9, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((T + 9, 8), 5.0, device="cuda")
    ws = torch.empty(msa.prefix_attention_workspace_bytes(600, T + 9, 8, 2, 1, w["max_q"], w["max_k"]), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _run(w, mask, out=out, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out[:T], got[0]) and torch.equal(lse[:T], got[1]) and (out[T:] == 5).all() and (lse[T:] == 5).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = msa.msa_tree_attention(w["q"], w["kv"], QS, KS, VS, SM, w["table"], w["cu_q"], w["cu_k"], mask, 1, w["max_q"], w["max_k"])
    graph.replay()
    assert torch.equal(o[:T], got[0]) and torch.equal(s[:T], got[1])


# ----------------------------------------------------------------- acceptance


def _walk(parents, drafts, chosen):
    path = [0]
    while True:
        c = [i for i in range(1, len(parents)) if parents[i] == path[-1] and drafts[i] == chosen[path[-1]]]
        if not c:
            return path
        path.append(c[0])


def _pools(layers, pages, heads, fp4, g):
    shape = (pages, heads, 2, 9216) if fp4 else (pages, heads, 128, 256)
    return [torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(layers)]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("lens,kind,agree", [([1], "chain", 1.0), ([256], "chain", 1.0), ([256], "two", 1.0), ([16, 1, 0, 40], "random", 0.8),
                                             ([64] * 9, "random", 0.9), ([255, 256, 100], "two", 0.97), ([5] * 40, "star", 0.5), ([30, 31], "random", 0.0)])
def test_accept(lens, kind, agree, fp4):
    r = np.random.RandomState(len(lens) + sum(lens))
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    heads, layers = (3, 5) if len(lens) < 9 else (2, 70)
    seqs = [n + int(r.randint(0, 300)) for n in lens]
    pages = [-(-s // 128) for s in seqs]
    perm = r.permutation(sum(pages) + 1)
    table = np.full((len(lens), max(max(pages), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    parents = [_parents(n, kind, r) for n in lens]
    drafts = [r.randint(0, 5 if kind == "star" else 1000, n) for n in lens]
    chosen = []
    for p, d, n in zip(parents, drafts, lens):
        c = r.randint(0, 1000, n)
        for i in range(n):
            kids = [j for j in range(n) if p[j] == i]
            if kids and r.rand() < agree:
                c[i] = d[kids[-1]]
        chosen.append(c)
    pools = _pools(layers, sum(pages) + 1, heads, fp4, g)
    want = [p.clone() for p in pools]
    most = max(lens)
    tokens, accepted, path = np.full((len(lens), most), -1), np.zeros(len(lens), int), np.full((len(lens), most), -1)
    for b, n in enumerate(lens):
        if not n:
            continue
        way = _walk(parents[b], drafts[b], chosen[b])
        accepted[b] = len(way) - 1
        path[b, :len(way)] = way
        tokens[b, :len(way)] = [drafts[b][i] for i in way[1:]] + [chosen[b][way[-1]]]
        src, dst = torch.tensor([seqs[b] - n + i for i in way]), torch.arange(seqs[b] - n, seqs[b] - n + len(way))
        page = torch.from_numpy(table[b]).long()
        for old, new in zip(pools, want):
            x = old.cpu()
            y = new.cpu()
            if fp4:
                for lo, size in ((0, 64), (8192, 8)):
                    u = x[..., lo:lo + 128 * size].reshape(*x.shape[:3], 128, size)
                    v = y[..., lo:lo + 128 * size].reshape(*x.shape[:3], 128, size).clone()
                    v[page[dst // 128], :, :, dst % 128] = u[page[src // 128], :, :, src % 128]
                    y[..., lo:lo + 128 * size] = v.reshape(*x.shape[:3], 128 * size)
            else:
                y[page[dst // 128], :, dst % 128] = x[page[src // 128], :, src % 128]
            new.copy_(y)
    status = i32([0])
    fn = msa.msa_tree_accept_nvfp4 if fp4 else msa.msa_tree_accept
    flat = lambda v: i32(np.concatenate(v).astype(int).tolist() + [0, 0])  # noqa: E731
    args = (flat(drafts), flat(parents), flat(chosen), cum(lens), cum(seqs), most)
    got = fn(*args)
    assert np.array_equal(got[0].cpu().numpy(), tokens) and np.array_equal(got[1].cpu().numpy(), accepted) and np.array_equal(got[2].cpu().numpy(), path)
    got = fn(*args, kv=pools, block_table=torch.from_numpy(table).cuda(), status=status)
    assert status.item() == 0
    assert np.array_equal(got[0].cpu().numpy(), tokens) and np.array_equal(got[1].cpu().numpy(), accepted) and np.array_equal(got[2].cpu().numpy(), path)
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_accept_takes_pools_in_each_form_and_tells_of_bad_ones():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    all_pools = torch.randint(0, 256, (3, 4, 2, 128, 256), generator=g, device="cuda", dtype=torch.uint8)
    table = i32([[2, 0]])
    # path 0, 2, 3: rows 122 + 2, 122 + 3 to 123, 124
    args = (i32([0, 8, 9, 7, 5]), i32([-1, 0, 0, 2, 9]), i32([9, 1, 7, 4, 4]), i32([0, 5]), i32([0, 127]), 5)
    want = all_pools.clone()
    want[:, 2, :, 123:125] = all_pools[:, 2, :, 124:126]
    status = i32([0])
    for kv in (all_pools.clone(), list(all_pools.clone()), all_pools.clone()[1].clone()):
        tokens, accepted, path = msa.msa_tree_accept(*args, kv=kv, block_table=table, status=status)
        assert tokens.tolist() == [[9, 7, 4, -1, -1]] and accepted.tolist() == [2] and path.tolist() == [[0, 2, 3, -1, -1]]
        got = torch.stack(kv) if isinstance(kv, list) else kv
        assert torch.equal(got, want if got.dim() == 5 else want[1])
    assert status.item() == msa.STATUS_BAD_TREE  # node 4's parent
    # a page that is none: nothing is moved there
    status.zero_()
    kv = all_pools.clone()
    msa.msa_tree_accept(*args, kv=kv, block_table=i32([[4, 0]]), status=status)
    assert status.item() == msa.STATUS_BAD_TREE | msa.STATUS_BAD_BLOCK and torch.equal(kv, all_pools)
    # a table too narrow, lengths that do not fit
    status.zero_()
    tokens, accepted, path = msa.msa_tree_accept(*args[:4], i32([0, 4]), 5, kv=kv, block_table=table, status=status)
    assert status.item() == msa.STATUS_BAD_SEQLENS and (tokens == -1).all() and accepted.item() == 0 and (path == -1).all()
    status.zero_()
    msa.msa_tree_accept(*args[:4], i32([0, 1000]), 5, kv=kv, block_table=table, status=status)
    assert status.item() & msa.STATUS_BAD_SEQLENS and torch.equal(kv, all_pools)


def test_accept_as_a_graph():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    start = torch.randint(0, 256, (2, 4, 2, 128, 256), generator=g, device="cuda", dtype=torch.uint8)
    kv, table = start.clone(), i32([[2, 0]])
    chosen = i32([9, 1, 7, 4, 4])
    args = (i32([0, 8, 9, 7, 5]), i32([-1, 0, 0, 2, 1]), chosen, i32([0, 5]), i32([0, 127]), 5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, accepted, path = msa.msa_tree_accept(*args, kv=kv, block_table=table)
    graph.replay()
    assert accepted.tolist() == [2] and torch.equal(kv[:, 2, :, 123:125], start[:, 2, :, 124:126])
    kv.copy_(start)
    chosen.copy_(i32([8, 5, 7, 4, 3]))
    graph.replay()
    assert tokens.tolist() == [[8, 5, 3, -1, -1]] and path.tolist() == [[0, 1, 4, -1, -1]]
    want = start.clone()
    want[:, 2, :, 124] = start[:, 2, :, 126]
    assert torch.equal(kv, want)
