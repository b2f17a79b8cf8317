"""Dense attention behind a shared prefix against attention in 64 bits.

Tolerance of the output, from the roundings: bf16 of the result (2^-8 of it),
f16 of each probability (2^-11 of it, so 2^-11 of A = sum p |v|), and fp32
sums over at most 10^4 keys in chains of a quarter of them (below 2^-12 of
A): |got - ref| <= 2^-8 |ref| + 2^-10 A.  The lse: the same sums give 2^-12,
each score c s - c m one fp32 rounding of at most 2^-23 of the largest."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

QS, KS, VS, SM = 0.0131, 0.0127, 0.0149, 128 ** -0.5


def _batch(hq, hkv, q_lens, own, prefix, seed=0, gain=1.0, spare=3):
    """Random E4M3 q and pool; request b has prefix pages and own[b] keys."""
    r = np.random.RandomState(seed)
    seqs = [prefix * 128 + n if q else n for n, q in zip(own, q_lens)]
    need = [max(0, -(-s // 128) - prefix) for s in seqs]
    pages = prefix + sum(need) + spare
    perm = r.permutation(pages).astype(np.int32)
    table = np.full((len(seqs), max(1, prefix + max(need))), -1, np.int32)
    at = prefix
    for b, n in enumerate(need):
        table[b, :prefix] = perm[:prefix]
        table[b, prefix:prefix + n] = perm[at:at + n]
        at += n
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kv = (torch.randn((pages, hkv, 128, 256), generator=g, device="cuda") / 0.013).to(torch.float8_e4m3fn)
    T = sum(q_lens)
    q = (gain * torch.randn((T, hq, 128), generator=g, device="cuda") / 0.013).clamp(-448, 448).to(torch.float8_e4m3fn)
    cu = lambda v: torch.from_numpy(np.concatenate([[0], np.cumsum(v)]).astype(np.int32)).cuda()  # noqa: E731
    return {"q": q, "kv": kv, "table": torch.from_numpy(table).cuda(), "cu_q": cu(q_lens), "cu_k": cu(seqs), "prefix": prefix,
            "max_q": max(q_lens), "max_k": max(max(seqs), prefix * 128, max(q_lens)), "q_lens": q_lens, "seqs": seqs}


def _run(w, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = msa.msa_prefix_attention(w["q"], w["kv"], QS, KS, VS, SM, w["table"], w["cu_q"], w["cu_k"], w["prefix"], w["max_q"], w["max_k"],
                                        status=status, **kw)
    torch.cuda.synchronize()
    return out, lse, status.item()


def _reference(w, left_out=()):
    """(out, A, lse) in 64 bits; left_out: physical pages whose keys do not count."""
    hq, hkv = w["q"].shape[1], w["kv"].shape[1]
    G = hq // hkv
    outs = []
    table = w["table"].long()
    at = 0
    q = w["q"].double() * (QS * KS * SM)
    for b, (n, m) in enumerate(zip(w["q_lens"], w["seqs"])):
        if not n:
            continue
        pages = table[b, :-(-m // 128)]
        there = torch.tensor([int(x) not in left_out and 0 <= int(x) < w["kv"].shape[0] for x in pages], device="cuda").repeat_interleave(128)[:m]
        x = w["kv"][pages.clamp(0, w["kv"].shape[0] - 1)].double().transpose(0, 1).reshape(hkv, -1, 256)[:, :m].repeat_interleave(G, 0)
        z = torch.einsum("thd,hkd->thk", q[at:at + n], x[..., :128])
        seen = there & (torch.arange(m, device="cuda") <= torch.arange(m - n, m, device="cuda")[:, None])
        z = torch.where(seen[:, None], z, -torch.inf)
        lse = torch.logsumexp(z, -1)
        p = torch.where(seen[:, None], torch.exp(z - lse[..., None]), 0.0)
        p = torch.where(torch.isneginf(lse)[..., None], torch.zeros_like(p), p)
        v = x[..., 128:]
        mask = seen[:, None, :, None].expand(n, hq, m, 1) if torch.isnan(v).any() else None
        if mask is None:
            o, a = torch.einsum("thk,hkd->thd", p, v), torch.einsum("thk,hkd->thd", p, v.abs())
        else:  # a key that is not seen has no part in the sum, whatever it holds
            vv = torch.where(mask, v[None].expand(n, hq, m, 128), 0.0)
            o, a = (p[..., None] * vv).sum(2), (p[..., None] * vv.abs()).sum(2)
        outs.append((o * VS, a * VS, lse))
        at += n
    return [torch.cat(x) for x in zip(*outs)]


def _compare(w, got, left_out=()):
    out, lse = got[0].double(), got[1].double()
    ref, a, ref_lse = _reference(w, left_out)
    assert torch.equal(torch.isnan(out), torch.isnan(ref)) and torch.equal(torch.isnan(lse), torch.isnan(ref_lse))
    err = (out - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -10 * a)
    assert not (err > 0).any(), (err.nan_to_num(-1).max().item(), err.nan_to_num(-1).argmax().item())
    inf = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), inf)
    ok = ~inf & ~torch.isnan(ref_lse)
    assert ((lse - ref_lse).abs()[ok] <= 2.0 ** -12 + 2.0 ** -20 * ref_lse.abs()[ok]).all()


CASES = [
    # hq, hkv, q_lens, own keys, prefix pages
    (8, 1, [1], [1], 0),
    (8, 1, [1], [128], 1),
    (8, 1, [1], [129], 3),
    (16, 2, [8] * 4, [8, 100, 128, 300], 5),
    (16, 2, [8] * 4, [1000, 2000, 3001, 4100], 0),
    (16, 2, [300], [300], 9),
    (16, 2, [257], [900], 0),
    (12, 4, [1, 0, 40, 129, 3], [1, 5, 41, 700, 128], 2),
    (1, 1, [200, 1], [200, 4000], 1),
    (128, 1, [3, 2], [10, 300], 2),
    (256, 2, [1, 5], [1, 5], 1),
    (5, 1, [26, 25, 51], [26, 200, 60], 3),
    (35, 7, [9, 2], [129, 257], 1),
    (4, 4, [1] * 70, [1 + 3 * i for i in range(70)], 2),
    (8, 2, [1] * 1100, [1 + i % 300 for i in range(1100)], 1),
    (16, 2, [16, 17, 32, 33, 48], [16, 145, 32, 161, 300], 4),
    (8, 1, [1], [9000], 0),
    (32, 8, [2] * 9, [9000 + 7 * i for i in range(9)], 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_64_bits(case):
    w = _batch(*CASES[case], seed=case)
    out, lse, status = _run(w)
    assert status == 0
    _compare(w, (out, lse))


@pytest.mark.parametrize("gain", [0.01, 6.0, 40.0])
def test_flat_and_peaked_scores(gain):
    # the running maximum grows by far more than the lag along the keys
    w = _batch(16, 2, [8, 3, 30], [700, 3, 1100], 7, seed=3, gain=gain)
    w["kv"].view(torch.uint8)  # ascending key sizes: later pages hold larger maxima
    kv = w["kv"].float()
    for i, page in enumerate(w["table"][2].tolist()):
        if page >= 0:
            kv[page, :, :, :128] *= 0.2 + 0.1 * i
    w["kv"] = kv.clamp(-448, 448).to(torch.float8_e4m3fn)
    out, lse, status = _run(w)
    assert status == 0
    _compare(w, (out, lse))


def test_scales_whose_product_vanishes():
    # scores below 2^-100: every key has the same weight; what is masked has none
    w = _batch(8, 2, [40, 2], [300, 4], 2, seed=12)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = msa.msa_prefix_attention(w["q"], w["kv"], 1e-30, 1e-25, VS, SM, w["table"], w["cu_q"], w["cu_k"], w["prefix"], w["max_q"], w["max_k"],
                                   status=status)
    assert status.item() == 0
    _compare(dict(w, q=torch.zeros_like(w["q"].view(torch.uint8)).view(torch.float8_e4m3fn)), got)


def test_prefix_equals_no_prefix():
    # the same keys, once as shared pages and once as every request's own
    w = _batch(16, 2, [8, 1, 40], [50, 300, 41], 6, seed=4)
    a = _run(w)
    w["prefix"] = 0
    b = _run(w)
    _compare(w, a[:2])
    _compare(w, b[:2])


def test_codes_behind_the_end_have_no_effect():
    # NaN codes in all pages that nothing uses and behind every request's end
    w = _batch(12, 4, [3, 130, 1], [5, 131, 129], 2, seed=5)
    want = _run(w)
    raw = w["kv"].view(torch.uint8).clone()
    used = torch.zeros(raw.shape[0], 128, dtype=torch.bool, device="cuda")
    for b, m in enumerate(w["seqs"]):
        for p in range(-(-m // 128)):
            used[w["table"][b, p], :min(128, m - p * 128)] = True
    raw = torch.where(used[:, None, :, None], raw, torch.full_like(raw, 0xFF))
    w["kv"] = raw.view(torch.float8_e4m3fn)
    got = _run(w)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_nan_reaches_only_rows_that_see_it():
    w = _batch(8, 2, [40, 2], [300, 4], 2, seed=6)
    raw = w["kv"].view(torch.uint8)
    t0, t1 = w["table"][0], w["table"][1]
    raw[t0[2 + 270 // 128], 0, 270 % 128, 128 + 5] = 0x7F   # V of request 0's own key 270: queries 270 and on, column 5
    raw[t0[2 + 290 // 128], 1, 290 % 128, 7] = 0xFF         # K of its key 290
    raw[t1[2], 1, 3, 128:] = 0x7F                            # V of request 1's last key
    out, lse, status = _run(w)
    assert status == 0
    _compare(w, (out, lse))
    assert torch.isnan(out[10, 0, 5]) and not torch.isnan(out[9]).any() and torch.isnan(lse[30, 4]) and not torch.isnan(out[40]).any()
    raw[t0[0], 1, 17, 128 + 100] = 0xFF                      # V of a shared key: every row of the head
    out, lse, _ = _run(w)
    _compare(w, (out, lse))
    assert torch.isnan(out[:, 4:, 100]).all() and not torch.isnan(out[:, :4, 100]).any()


def test_bad_pages_are_left_out():
    w = _batch(8, 2, [2, 3], [200, 300], 3, seed=7)
    w["table"][0, 3] = w["kv"].shape[0]    # own page of request 0
    w["table"][:, 1] = -5                  # a shared one
    w["table"][1, 5] = -1                  # the last of request 1: its queries see no own key of it
    out, lse, status = _run(w)
    assert status == msa.STATUS_BAD_BLOCK
    _compare(w, (out, lse))
    w = _batch(8, 2, [2], [130], 0, seed=7)
    w["table"][:] = -1
    out, lse, status = _run(w)
    assert status == msa.STATUS_BAD_BLOCK and not out.any() and torch.isneginf(lse).all()


def test_bad_lengths_give_empty_rows():
    base = _batch(8, 2, [4, 4], [10, 300], 2, seed=8)
    for name, cu_q, cu_k in (("inside the prefix", [0, 4, 8], [0, 259, 700]), ("more queries than keys", [0, 4, 8], [0, 300, 303]),
                             ("descending", [0, 9, 8], [0, 300, 700]), ("past max_seqlen_k", [0, 4, 8], [0, 300, 1700]),
                             ("more than T", [0, 4, 9], [0, 300, 700]), ("not from 0", [1, 4, 8], [0, 300, 700])):
        w = dict(base, cu_q=torch.tensor(cu_q, dtype=torch.int32).cuda(), cu_k=torch.tensor(cu_k, dtype=torch.int32).cuda())
        out, lse, status = _run(w)
        assert status == msa.STATUS_BAD_SEQLENS and not out.any() and torch.isneginf(lse).all(), name


def test_rows_behind_the_batch_are_left_as_they_were():
    w = _batch(16, 2, [8, 0, 3], [100, 0, 300], 2, seed=9)
    want = _run(w)
    pad = torch.cat((w["q"].view(torch.uint8), torch.full((5, 16, 128), 0x7F, dtype=torch.uint8, device="cuda"))).view(torch.float8_e4m3fn)
    out = torch.full((16, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((16, 16), 7.0, device="cuda")
    # requests without queries, their lengths 0, at the end of the batch too
    w = dict(w, q=pad, cu_q=torch.cat((w["cu_q"], w["cu_q"][-1:])), cu_k=torch.cat((w["cu_k"], w["cu_k"][-1:])),
             table=torch.cat((w["table"], torch.full_like(w["table"][:1], -1))))
    got = _run(w, out=out, lse=lse)
    assert got[2] == 0 and torch.equal(out[:11], want[0]) and torch.equal(lse[:11], want[1])
    assert (out[11:] == 7.0).all() and (lse[11:] == 7.0).all()
    none = dict(w, cu_q=torch.zeros_like(w["cu_q"]))
    out.fill_(3.0)
    assert _run(none, out=out, lse=lse)[2] == 0 and (out == 3.0).all()


def test_graph_streams_and_repeats():
    w = _batch(16, 2, [8] * 6, [300 * (i + 1) for i in range(6)], 20, seed=10)
    want = _run(w)
    for _ in range(3):
        again = _run(w)
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    other = _batch(16, 2, [8] * 6, [200 * (i + 1) for i in range(6)], 11, seed=11)
    want2 = _run(other)
    # two calls at once on two streams, each with a workspace of its own
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for x, s in ((w, a), (other, b)):
            got.append(msa.msa_prefix_attention(x["q"], x["kv"], QS, KS, VS, SM, x["table"], x["cu_q"], x["cu_k"], x["prefix"], x["max_q"], x["max_k"], stream=s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], (want, want2)[i % 2][0]) and torch.equal(g[1], (want, want2)[i % 2][1])
    # captured; the lengths and inputs may change between replays
    need = msa.prefix_attention_workspace_bytes(6, 48, 16, 2, 20, 8, w["max_k"])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    cu_k = w["cu_k"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.msa_prefix_attention(w["q"], w["kv"], QS, KS, VS, SM, w["table"], w["cu_q"], cu_k, 20, 8, w["max_k"], workspace=ws, out=out, lse=lse)
    for shorter in (0, 37, 0):
        seqs = [s - shorter for s in w["seqs"]]
        cu_k.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(seqs)]).astype(np.int32)))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        _compare(dict(w, seqs=seqs), (out, lse))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_more_tiles_than_a_plan_round():
    # 128 query heads a KV head: 2 tokens a tile, 550 own and 550 shared tiles
    w = _batch(128, 1, [700, 400], [700, 450], 1, seed=14)
    out, lse, status = _run(w)
    assert status == 0
    _compare(w, (out, lse))


def test_pages_beyond_32_bits_and_an_unaligned_output():
    w = _batch(16, 2, [8, 3], [300, 200], 3, seed=15)
    want = _run(w)
    n, high = w["kv"].shape[0], 70000  # 4.6 GB
    pool = torch.empty((high, 2, 128, 256), dtype=torch.uint8, device="cuda")
    pool[high - n:] = w["kv"].view(torch.uint8)
    table = torch.where(w["table"] >= 0, w["table"] + high - n, w["table"])
    room = torch.zeros(11 * 16 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    out = room[4:-4].view(11, 16, 128)  # on 8 bytes
    got = _run(dict(w, kv=pool.view(torch.float8_e4m3fn), table=table), out=out)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not room[:4].any() and not room[-4:].any()


def test_short_wait_limit_expires_and_the_next_call_is_clean():
    # a limit below a page load's latency: a wait runs out, the call returns
    # with the status bit, and the next one on the same workspace is exact
    lib = msa.load()
    w = _batch(16, 2, [8] * 4, [1000, 2000, 3001, 4100], 30, seed=13)
    need = msa.prefix_attention_workspace_bytes(4, 32, 16, 2, 30, 8, w["max_k"])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = _run(w, workspace=ws)
    assert want[2] == 0
    try:
        assert lib.msa_test_set_wait_limit_ns(300) == 0
        assert _run(w, workspace=ws)[2] & msa.STATUS_TIMEOUT
    finally:
        lib.msa_test_set_wait_limit_ns(0)
    got = _run(w, workspace=ws)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("low", [0, 1])
@pytest.mark.parametrize("hq,hkv,q_lens,own,prefix", [
    (16, 2, [1], [5000], 0),             # one token over many CTAs
    (16, 2, [8] * 400, [300] * 400, 0),  # whole tiles to a CTA: the two streams' halves
    (16, 2, [8] * 4, [200] * 4, 6),      # shared pages beside own ones
    (4, 4, [150], [700], 0),             # pages that some rows see in part
    (8, 1, [40], [41], 2),
])
def test_nan_of_keys_without_weight(hq, hkv, q_lens, own, prefix, low):
    # the keys of one page lie some 800 powers of two below the others: their
    # weight is 0 in fp32 wherever the page is merged, and a NaN there is one
    w = _batch(hq, hkv, q_lens, own, prefix, seed=16)
    w["q"] = torch.full(w["q"].shape, 384.0, device="cuda").to(torch.float8_e4m3fn)
    kv = w["kv"].float()
    kv[..., :128] = 320.0
    kv[w["table"][:, low].long(), ..., :128] = -320.0
    w["kv"] = kv.to(torch.float8_e4m3fn)
    clean = _run(w)
    assert clean[2] == 0
    _compare(w, clean[:2])
    raw, page = w["kv"].view(torch.uint8), w["table"][-1, low].item()
    raw[page, 0, 20, 128 + 5] = 0x7F        # V of one of its keys: column 5
    out, lse, status = _run(w)
    assert status == 0
    _compare(w, (out, lse))
    assert torch.isnan(out[-1, 0, 5]) and not torch.isnan(lse).any()
    raw[page, hkv - 1, 9, 7] = 0xFF         # K of another: the rows
    out, lse, status = _run(w)
    assert status == 0
    _compare(w, (out, lse))
    assert torch.isnan(out[-1, -1]).all() and torch.isnan(lse[-1, -1])


def test_bound_far_above_the_lengths():
    # a batch under the largest bound: 32 short requests, 2^23 pages a row of the table
    w = _batch(16, 2, [1] * 30 + [40, 2], [1 + 20 * i for i in range(30)] + [300, 7], 0, seed=17)
    want = _run(w)
    table = torch.full((32, 2 ** 23), -1, dtype=torch.int32, device="cuda")
    table[:, :w["table"].shape[1]] = w["table"]
    got = _run(dict(w, table=table, max_k=2 ** 30))
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_long_rows_of_one_page():
    # 64 requests of 2^21 keys each, all in one page: the softmax over it,
    # whatever the number of its copies
    w = _batch(16, 1, [1] * 64, [128] * 64, 0, seed=18)
    want = _reference(w)
    pages, P = w["table"][:, 0].clone(), 2 ** 14
    table = pages[:, None].expand(64, P).contiguous()
    cu_k = torch.arange(65, dtype=torch.int32, device="cuda") * (128 * P)
    out, lse, status = _run(dict(w, table=table, cu_k=cu_k, max_k=128 * P))
    assert status == 0
    err = (out.double() - want[0]).abs() - (2.0 ** -8 * want[0].abs() + 2.0 ** -10 * want[1])
    assert not (err > 0).any()
    assert ((lse.double() - want[2] - np.log(P)).abs() <= 2.0 ** -11).all()


@pytest.mark.parametrize("n,own", [(8, [40000 + 100 * i for i in range(8)]), (1, [100 + 800 * i // 512 for i in range(512)])])
def test_a_nan_does_not_slow_the_rest_of_the_batch(n, own):
    # a NaN among the V of the first request's last page: only the page that
    # holds it is looked through, not every page that follows
    w = _batch(16, 2, [n] * len(own), own, 0, seed=19)
    dirty = dict(w, kv=w["kv"].view(torch.uint8).clone())
    dirty["kv"][w["table"][0, (w["seqs"][0] - 1) // 128], :, (w["seqs"][0] - 1) % 128, 128 + 9] = 0x7F
    dirty["kv"] = dirty["kv"].view(torch.float8_e4m3fn)
    out, lse, status = _run(dirty)
    assert status == 0 and torch.isnan(out[n - 1, :, 9]).all() and not torch.isnan(out[n:]).any() and not torch.isnan(lse).any()
    took = {}
    for name, x in (("clean", w), ("dirty", dirty)):
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            msa.msa_prefix_attention(x["q"], x["kv"], QS, KS, VS, SM, x["table"], x["cu_q"], x["cu_k"], 0, x["max_q"], x["max_k"])
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took[name] = min(times)
    print(took)
    assert took["dirty"] < 2 * took["clean"] + 0.1, took
