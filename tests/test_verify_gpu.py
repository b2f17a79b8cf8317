"""Draft verification against plain Python integers: the accept test in 64
bits, weights in whole steps of 2^-44, the token by their exact cumulated
sums.  Everything is a whole number, so results are equal."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

TYPES = (torch.float32, torch.bfloat16, torch.float16)


def _weights(p, q):
    with np.errstate(invalid="ignore"):
        w = np.nan_to_num(p - q, nan=0.0, posinf=1.0)  # fp32
    return np.floor(np.clip(w, 0, 1).astype(np.float64) * 2.0 ** 44).astype(np.uint64)


def _pick(w, u):
    cut = np.cumsum(w, dtype=np.uint64)
    total = int(cut[-1])
    if total == 0:
        return None
    x = 0 if not u > 0 else min(int(float(u) * 2 ** 31), 2 ** 31 - 1)
    return int(np.searchsorted(cut, np.uint64(x * total >> 31), side="right"))


def _reference(target, draft, drafts, u, counts):
    B, n, V = target.shape
    tokens, accepted = np.full((B, n), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        most = n - 1 if counts is None else min(max(int(counts[b]), 0), n - 1)
        a = 0
        while a < most:
            x = int(drafts[b, a])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, a, x])
            if not float(u[b, a]) * q < float(target[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        p = target[b, a]
        q = np.zeros(V, np.float32)
        if a < most:
            if draft is not None:
                q = draft[b, a]
            elif 0 <= drafts[b, a] < V:
                q[drafts[b, a]] = np.inf
        t = _pick(_weights(p, q), u[b, -1])
        if t is None:
            t = _pick(_weights(p, np.zeros(V, np.float32)), u[b, -1])
        tokens[b, a] = -1 if t is None else t
        accepted[b] = a
    return tokens, accepted


def _check(target, draft, drafts, u, counts=None):
    got = msa.msa_verify(target, drafts, u, draft_probs=draft, num_drafts=counts)
    cpu = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    want = _reference(cpu(target), cpu(draft), drafts.cpu().numpy(), u.cpu().numpy(), None if counts is None else counts.cpu().numpy())
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    return want


def _inputs(B, k, V, dtype, seed, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = 3 * torch.randn((B, k + 1, V), generator=g, device="cuda")
    y = z[:, :k] + torch.randn((B, k, V), generator=g, device="cuda")
    target, draft = torch.softmax(z, -1).to(dtype), torch.softmax(y, -1).to(dtype)
    drafts = torch.multinomial(torch.softmax(y, -1).reshape(B * k, V), 1, generator=g).reshape(B, k).int() if k else \
        torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    u = torch.rand((B, k + 1), generator=g, device="cuda")
    if pad:  # rows of a padded vocabulary
        wide = torch.full((B, k + 1, V + pad), 9.0, dtype=dtype, device="cuda")
        wide[..., :V] = target
        target = wide[..., :V]
    return target, draft, drafts, u


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("B,k,V,pad", [(1, 0, 1, 0), (2, 1, 2, 0), (3, 2, 31, 0), (5, 7, 1000, 0), (4, 3, 1000, 24), (70, 3, 257, 7),
                                       (2, 31, 4099, 0), (3, 2, 65536, 0), (2, 1, 200003, 0), (1, 1, 524287, 1)])
def test_matches_integers(B, k, V, pad, dtype):
    target, draft, drafts, u = _inputs(B, k, V, dtype, 7 * V + k, pad)
    counts = torch.randint(-1, k + 2, (B,), dtype=torch.int32, generator=torch.Generator().manual_seed(V)).cuda()
    for d in (draft, None):
        _check(target, d, drafts, u)
        _check(target, d, drafts, u, counts)


def test_edges():
    V, k = 40, 4
    target, draft, drafts, u = _inputs(6, k, V, torch.float32, 3)
    drafts[0, 0], drafts[1, 1], drafts[2, 0] = -1, V, 2 ** 31 - 1
    u[3] = 0.0
    target[3, 0, drafts[3, 0].item()] = 0.0    # 0 < 0: falls
    draft[4, 0] = 0.0                          # any p > 0 stands
    u[4, -1] = float(np.nextafter(np.float32(1), np.float32(0)))
    u[5] = float("nan")
    _check(target, draft, drafts, u)
    # NaN, infinite and negative entries have no weight (infinite: all of it)
    target[0, 0, 5], target[0, 0, 6], target[0, 0, 7] = float("nan"), -1.0, float("inf")
    draft[1, 1, 3] = float("nan")
    _check(target, draft, drafts, u)
    # nothing left of p - q: drawn from p; p without any probability: -1
    t2, d2 = target.clone(), draft.clone()
    t2[2, 0] = 0.5 * torch.softmax(torch.arange(V, device="cuda").float() / 9, -1)
    d2[2, 0] = 1.0
    t2[0, 0] = 0.0
    t2[5] = 0.0
    want = _check(t2, d2, drafts, u)
    assert want[0][0, 0] == -1 and want[0][2, 0] >= 0


def test_certain_draft_refused_where_nothing_else_has_probability():
    # p has weight at the draft alone, and too little of it to stand: without
    # the draft nothing is left, so the token is drawn from p, the draft again
    for V in (7, 5003):
        target = torch.zeros((2, 2, V), device="cuda")
        target[:, 0, 5], target[:, 1, 1] = 0.3, 1.0
        drafts = torch.full((2, 1), 5, dtype=torch.int32, device="cuda")
        u = torch.tensor([[0.9, 0.5], [0.2, 0.5]], device="cuda")
        want = _check(target, None, drafts, u)
        assert want[0].tolist() == [[5, -1], [5, 1]] and want[1].tolist() == [0, 1]


def test_uniforms_reproduce_the_distribution():
    # N evenly spread uniforms over one row: each token is drawn N p times,
    # up to one either side of its interval's two ends
    N, V = 4096, 300
    target, draft, drafts, u = _inputs(1, 1, V, torch.float32, 9)
    target, draft, drafts = (t.expand(N, *t.shape[1:]).contiguous() for t in (target, draft, drafts))
    even = (torch.arange(N, device="cuda") + 0.5) / N
    u = torch.stack((torch.full_like(even, 0.999999), even), 1)
    target[:, 0, drafts[0, 0].item()] = 0.0  # always falls
    tokens, accepted = msa.msa_verify(target, drafts, u, draft_probs=draft)
    assert not accepted.any()
    w = (target[0, 0].double() - draft[0, 0].double()).clamp(min=0)
    want = w / w.sum() * N
    got = torch.bincount(tokens[:, 0].long(), minlength=V).double()
    assert ((got - want).abs() <= 1.001).all()


def _greedy_reference(x, drafts, counts):
    B, n, V = x.shape
    tokens, accepted = np.full((B, n), -1, np.int32), np.zeros(B, np.int32)

    def best(row):
        if np.isnan(row).all():
            return -1
        return int(np.flatnonzero(row == np.nanmax(row))[0])

    for b in range(B):
        most = n - 1 if counts is None else min(max(int(counts[b]), 0), n - 1)
        a = 0
        while a < most and drafts[b, a] >= 0 and best(x[b, a]) == drafts[b, a]:
            tokens[b, a] = drafts[b, a]
            a += 1
        tokens[b, a] = best(x[b, a])
        accepted[b] = a
    return tokens, accepted


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("B,k,V,pad", [(1, 0, 1, 0), (3, 1, 2, 0), (4, 3, 31, 0), (9, 7, 1000, 0), (5, 7, 4099, 5), (3, 31, 257, 0), (40, 2, 65536, 0),
                                       (2, 3, 200003, 0)])
def test_greedy_matches(B, k, V, pad, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(V + k)
    # coarse values: many ties for the best
    x = torch.randint(-40, 40, (B, k + 1, V + pad), generator=g, device="cuda").to(dtype)[..., :V]
    first = torch.where(x.float() == x.float().amax(-1, keepdim=True), torch.arange(V, device="cuda"), V).amin(-1)[:, :k].int()
    miss = torch.rand((B, k), generator=g, device="cuda") < 0.2
    drafts = torch.where(miss, torch.randint(0, V, (B, k), generator=g, device="cuda", dtype=torch.int32), first).contiguous()
    counts = torch.randint(0, k + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    for c in (None, counts):
        got = msa.msa_verify_greedy(x, drafts, num_drafts=c)
        want = _greedy_reference(x.float().cpu().numpy(), drafts.cpu().numpy(), None if c is None else c.cpu().numpy())
        assert np.array_equal(got[1].cpu().numpy(), want[1])
        assert np.array_equal(got[0].cpu().numpy(), want[0])


def test_greedy_edges():
    inf, nan = float("inf"), float("nan")
    x = torch.full((7, 3, 5000), -inf, device="cuda")
    drafts = torch.zeros((7, 2), dtype=torch.int32, device="cuda")
    x[1, 0, 4000] = x[1, 0, 100] = inf          # a tie of infinities: the lower one
    drafts[1, 0] = 100
    x[2, 0] = nan                               # nothing but NaN
    x[3, 0, 3], x[3, 0, 4] = nan, 2.0           # NaN is never the best
    drafts[3, 0] = 3
    x[4, 0] = -1.0
    x[4, 0, 4999], x[4, 0, 17] = 0.0, -0.0      # +0 and -0 are equal
    drafts[4, 0] = 17
    drafts[5, 0], drafts[6, 1] = -1, 5000       # not tokens
    got = msa.msa_verify_greedy(x, drafts)
    want = _greedy_reference(x.cpu().numpy(), drafts.cpu().numpy(), None)
    assert np.array_equal(got[1].cpu().numpy(), want[1]) and np.array_equal(got[0].cpu().numpy(), want[0])
    assert want[0][2, 0] == -1 and want[1][4] >= 1


def test_graph_and_other_stream():
    target, draft, drafts, u = _inputs(6, 3, 3001, torch.bfloat16, 5)
    want = msa.msa_verify(target, drafts, u, draft_probs=draft)
    best = msa.msa_verify_greedy(target, drafts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = msa.msa_verify(target, drafts, u, draft_probs=draft, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    tokens = torch.empty_like(want[0]), torch.empty_like(want[0])
    accepted = torch.empty_like(want[1]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.msa_verify(target, drafts, u, draft_probs=draft, tokens=tokens[0], accepted=accepted[0])
        msa.msa_verify_greedy(target, drafts, tokens=tokens[1], accepted=accepted[1])
    for _ in range(2):
        for t in tokens + accepted:
            t.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens[0], want[0]) and torch.equal(accepted[0], want[1])
        assert torch.equal(tokens[1], best[0]) and torch.equal(accepted[1], best[1])


@pytest.mark.parametrize("B,k,V", [(700, 3, 1), (900, 2, 5), (600, 7, 64), (500, 3, 4096), (160, 2, 32000)])
def test_batches_that_fill_every_sm(B, k, V):
    # clusters that start late beside ones that run already, the smallest rows
    # (most CTAs have no part of them, and reach the exchange of the totals at
    # once) and rows of whole 16-byte pieces
    target, draft, drafts, u = _inputs(B, k, V, torch.float32, B + V)
    busy = torch.cuda.Stream()
    a = torch.randn((4096, 4096), device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        for _ in range(4):
            a @ a
    want = _check(target, draft, drafts, u)
    again = [msa.msa_verify(target, drafts, u, draft_probs=draft) for _ in range(20)]
    torch.cuda.synchronize()
    for tokens, accepted in again:
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])
    _check(target, None, drafts, u)


def _exact_pick(w, u):
    """The lowest v whose cumulated weight exceeds floor(u total), u taken exactly."""
    cut = np.cumsum(w, dtype=np.uint64)
    num, den = float(u).as_integer_ratio()
    return int(np.searchsorted(cut, np.uint64(num * int(cut[-1]) // den), side="right"))


@pytest.mark.parametrize("V", [1000, 4099, 200003])
def test_small_uniforms_count_to_their_last_bit(V):
    # uniforms far below 2^-7, whose last bits lie below 2^-31; fine weights at
    # the row's start, so that these bits choose the token
    B = 64
    r = np.random.RandomState(V)
    target = torch.zeros((B, 1, V), device="cuda")
    target[:, :, :300] = torch.from_numpy(np.ldexp(r.rand(B, 1, 300).astype(np.float32), -36)).cuda()
    target[:, 0, -1] = 1.0
    sig = r.randint(2 ** 23, 2 ** 24, B) | 1
    u = np.ldexp(sig.astype(np.float32), -24 - r.randint(28, 36, B)).astype(np.float32)
    u[:3] = 2.0 ** -31, np.nextafter(np.float32(2.0 ** -30), np.float32(0)), 2.0 ** -149
    tokens, accepted = msa.msa_verify(target, torch.zeros((B, 0), dtype=torch.int32, device="cuda"), torch.from_numpy(u[:, None]).cuda())
    want = [_exact_pick(_weights(target[b, 0].cpu().numpy(), np.zeros(V, np.float32)), u[b]) for b in range(B)]
    assert len(set(want)) > 10
    assert tokens[:, 0].tolist() == want and not accepted.any()
    # ordinary uniforms with low bits (below 2^-7), over a spread row
    target = torch.softmax(2 * torch.from_numpy(r.randn(B, 1, V)).float(), -1).cuda()
    u = np.ldexp(sig.astype(np.float32), -24 - r.randint(0, 20, B)).astype(np.float32)
    tokens, _ = msa.msa_verify(target, torch.zeros((B, 0), dtype=torch.int32, device="cuda"), torch.from_numpy(u[:, None]).cuda())
    want = [_exact_pick(_weights(target[b, 0].cpu().numpy(), np.zeros(V, np.float32)), u[b]) for b in range(B)]
    assert tokens[:, 0].tolist() == want


def test_accepted_in_place_of_num_drafts():
    # drafts that all fall: a number of drafts read after `accepted` replaced
    # it would take the row behind them for theirs
    for B, V in ((400, 3), (200, 5003)):
        target, draft, drafts, u = _inputs(B, 5, V, torch.float32, B)
        target[:, 0].scatter_(1, drafts[:, :1].long(), 0.0)
        counts = torch.randint(0, 6, (B,), dtype=torch.int32, generator=torch.Generator().manual_seed(V)).cuda()
        want = _check(target, draft, drafts, u, counts)
        best = msa.msa_verify_greedy(target, drafts, num_drafts=counts)
        for _ in range(5):
            own = counts.clone()
            tokens, accepted = msa.msa_verify(target, drafts, u, draft_probs=draft, num_drafts=own, accepted=own)
            assert accepted is own and np.array_equal(own.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[0])
            own = counts.clone()
            tokens, _ = msa.msa_verify_greedy(target, drafts, num_drafts=own, accepted=own)
            assert torch.equal(own, best[1]) and torch.equal(tokens, best[0])
        # and one request's tokens over its drafts
        for b in (0, 1):
            room = torch.cat((drafts[b], drafts[b, :1]))
            msa.msa_verify(target[b:b + 1], room[:5].view(1, 5), u[b:b + 1], draft_probs=draft[b:b + 1], num_drafts=counts[b:b + 1], tokens=room.view(1, 6))
            assert np.array_equal(room.cpu().numpy(), want[0][b])


def test_certain_drafts_that_are_no_tokens():
    for V in (40, 5003, 200003):
        target, _, drafts, u = _inputs(8, 2, V, torch.float32, V)
        drafts[0, 0], drafts[1, 0], drafts[2, 0] = -2 ** 31, 2 ** 31 - 1, -1
        drafts[3, 0], drafts[4, 0], drafts[5, 0], drafts[6, 1] = V, -2 ** 31 + 1, -2 ** 31 + 4096, -2 ** 31 + V
        want = _check(target, None, drafts, u)
        assert not want[1][:6].any()
