"""Log probabilities, ranks, entropies and best alternatives against 64 bits.

Tolerance of the sums, from the roundings, with n = ceil(V / 512) + 16 additions
in the longest chain (256 threads, two sums each, their merge): each e^d is off
by less than 2^-21 of itself plus 2^-23 |d| (d, its product with log2 e and the
power), and p |d| < 1 for any term, so l and s are off by less than (n 2^-24 +
2^-20) of l (1 + the mean |d|).  The mean |d| is the entropy and log l at most,
below log V < 14."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _reference(x, tokens, top):
    """x fp64 [T, V] without NaN or +inf."""
    T, V = x.shape
    z = x - x.amax(-1, keepdim=True)  # (first: beside 3e38 the sum's logarithm would be lost)
    z = z - z.exp().sum(-1, keepdim=True).log()
    z = torch.where(torch.isnan(z), -torch.inf, z)  # a row of -inf
    ok = (tokens >= 0) & (tokens < V)
    at = tokens.long().clamp(0, V - 1)[:, None]
    logprob = torch.where(ok, z.gather(1, at)[:, 0], -torch.inf)
    mine = x.gather(1, at)
    rank = ((x > mine) | ((x == mine) & (torch.arange(V, device="cuda") < at))).sum(-1)
    p = z.exp()
    entropy = -torch.where(p > 0, p * z, 0.0).sum(-1)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    best = torch.full((T, top), -1, device="cuda", dtype=torch.long)
    best[:, :order.shape[1]] = order
    value = torch.where(best >= 0, z.gather(1, best.clamp(min=0)), -torch.inf)
    return logprob, torch.where(ok, rank, -1), entropy, best, value


def _check(x, tokens, top):
    T, V = x.shape
    logprob, rank, entropy, best, value = msa.msa_logprobs(x, tokens, top=top)
    a, b, c, d, e = _reference(x.double(), tokens, top)
    assert torch.equal(rank.long(), b) and torch.equal(d, best.long())
    H = np.log(V) + 1
    tol = (1 + H) * ((V / 512 + 17) * 2.0 ** -24 + 2.0 ** -20)
    for got, want in ((logprob, a), (value, e)):
        assert got.dtype is torch.float32 and torch.equal(torch.isinf(got), torch.isinf(want)) and not torch.isnan(got).any()
        fine = ~torch.isinf(want)
        err = (got.double() - want).abs()[fine] - 2.0 ** -22 * want.abs()[fine]
        assert not (err > tol).any(), err.max().item() / tol
    err = (entropy.double() - c).abs()
    assert not (err > 2 * tol * (1 + H)).any(), err.max().item() / tol


SIZES = [(1, 1), (3, 2), (2, 7), (5, 31), (1, 255), (4, 256), (3, 257), (2, 513), (7, 1000), (16, 4097), (1, 32000), (40, 50257), (700, 3000), (5, 131072),
         (76, 65537), (153, 20000), (2, 200003), (305, 9001), (1, 2 ** 19 - 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_matches_64_bits(T, V, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(T * 7 + V)
    x = (3 * torch.randn((T, V), generator=g, device="cuda")).to(dtype)
    tokens = torch.randint(-1, V + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    for top in (0, 1, 5, 20, 32):
        _check(x, tokens, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(2, 40), (3, 5003), (8, 131072), (400, 30001)])
def test_ties_and_orders(T, V, dtype):
    """Rows that are hard to choose from: all equal, two levels, few levels, ascending, descending, one peak, +0 beside -0."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    at = torch.arange(V, device="cuda")
    rows = [torch.zeros(V, device="cuda"), (at % 2).float(), (torch.rand(V, generator=g, device="cuda") * 4).floor(), at / V * 20, -at / V * 20,
            (at == V - 1).float() * 60000, torch.where(at % 3 == 0, 0.0, -0.0), (at >= V - 40).float(), -((at // 300) % 50).float()]
    x = torch.stack([rows[i % len(rows)] for i in range(max(T, len(rows)))]).to(dtype)
    tokens = torch.randint(0, V, (x.shape[0],), generator=g, device="cuda", dtype=torch.int32)
    for top in (1, 20, 32):
        _check(x, tokens, top)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_values(dtype):
    """-inf and the type's lowest value, up to whole rows of them."""
    V = 3001
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((6, V), generator=g, device="cuda").to(dtype)
    low = torch.finfo(dtype).min
    x[0, 10:] = -torch.inf  # fewer values than are asked for
    x[1, 7:] = low
    x[2] = low
    x[3, :2990] = -torch.inf
    x[4] = -torch.inf
    x[5, ::2] = low
    x[5, 1::4] = -torch.inf
    tokens = torch.tensor([3, 5, 2999, 7, 0, 0], dtype=torch.int32, device="cuda")
    _check(x, tokens, 32)
    logprob, rank, entropy, best, value = msa.msa_logprobs(x, tokens, top=3)
    assert logprob[4] == -torch.inf and entropy[4] == 0 and best[4].tolist() == [0, 1, 2] and (value[4] == -torch.inf).all()
    assert entropy[2].item() == pytest.approx(np.log(V), rel=1e-5)


def test_nan_and_infinity():
    V = 2000
    x = torch.linspace(-3, 3, V, device="cuda").repeat(4, 1)
    x[0, 100] = torch.nan
    x[1, 50] = torch.inf
    x[2] = torch.nan
    x[3, 5:] = torch.nan
    tokens = torch.tensor([100, 50, 3, 2], dtype=torch.int32, device="cuda")
    logprob, rank, entropy, best, value = msa.msa_logprobs(x, tokens, top=7)
    assert torch.isnan(logprob).all() and torch.isnan(entropy).all()
    assert rank.tolist() == [-1, 0, -1, 2]
    assert best[0].tolist() == list(range(V - 1, V - 8, -1)) and best[1].tolist()[:2] == [50, V - 1]
    assert best[2].tolist() == [-1] * 7 and best[3].tolist() == [4, 3, 2, 1, 0, -1, -1]
    assert torch.isnan(value[0]).all() and (value[2] == -torch.inf).all()


def test_large_logits_keep_their_accuracy():
    x = (1e4 + 3 * torch.randn((4, 5000), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)))
    _check(x, torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda"), 5)
    _check(x - 3e4, torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda"), 5)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_and_given_outputs(dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    room = (3 * torch.randn((9, 1237), generator=g, device="cuda")).to(dtype)
    x = room[:, 5:5 + 1111]
    tokens = torch.arange(9, dtype=torch.int32, device="cuda")
    _check(x, tokens, 20)
    _check(room[:1].expand(9, -1), tokens, 4)
    outs = {"logprobs": torch.zeros(9, device="cuda"), "ranks": torch.zeros(9, dtype=torch.int32, device="cuda"), "entropy": torch.zeros(9, device="cuda"),
            "top_tokens": torch.zeros((9, 4), dtype=torch.int32, device="cuda"), "top_logprobs": torch.zeros((9, 4), device="cuda")}
    want = msa.msa_logprobs(x, tokens, top=4)
    got = msa.msa_logprobs(x, tokens, top=4, **outs)
    assert all(a is b for a, b in zip(got, outs.values())) and all(torch.equal(a, b) for a, b in zip(got, want))
    none = msa.msa_logprobs(x, top=4)
    assert none[0] is None and none[1] is None and all(torch.equal(a, b) for a, b in zip(none[2:], want[2:]))
    empty = msa.msa_logprobs(x[:0], tokens[:0], top=2)
    assert [tuple(t.shape) for t in empty] == [(0,), (0,), (0,), (0, 2), (0, 2)]


def test_rows_past_32_bits():
    """A batch whose last rows lie more than 2^32 values behind the first."""
    x = torch.zeros((8300, 524000), dtype=torch.bfloat16, device="cuda")
    x[-1, 123456] = 5
    x[-2, 7] = 3
    tokens = torch.full((8300,), 7, dtype=torch.int32, device="cuda")
    logprob, rank, entropy, best, _ = msa.msa_logprobs(x, tokens, top=2)
    assert best[-1].tolist() == [123456, 0] and best[-2].tolist() == [7, 0] and best[0].tolist() == [0, 1]
    assert rank[-2:].tolist() == [0, 8] and rank[0] == 7
    assert (entropy[:8298].double() - np.log(524000)).abs().max() < 1e-3


def test_graph_and_other_stream():
    x = torch.randn((33, 40000), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    tokens = torch.arange(33, dtype=torch.int32, device="cuda")
    want = msa.msa_logprobs(x, tokens, top=20)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = msa.msa_logprobs(x, tokens, top=20, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = msa.msa_logprobs(x, tokens, top=20)
    for t in got:
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,V,dtype", [(24, 70001, torch.float32), (100, 40000, torch.float16), (64, 131072, torch.bfloat16), (152, 65535, torch.float16),
                                       (200, 131071, torch.bfloat16), (300, 50000, torch.float32), (500, 50001, torch.float32), (600, 70000, torch.bfloat16),
                                       (513, 33000, torch.float16), (1000, 65537, torch.bfloat16), (1300, 40001, torch.float32), (2500, 5001, torch.bfloat16)])
def test_numbers_of_rows(T, V, dtype):
    """Rows from a few to many rounds of the GPU's places: other CTAs, and other numbers of them a row."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + V)
    x = torch.randn((T, V), generator=g, device="cuda").to(dtype)
    x[T // 2] = 1.0  # equal values are chosen another way
    tokens = torch.randint(-1, V + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    for top in (3, 32):
        _check(x, tokens, top)


@pytest.mark.parametrize("T,V,dtype", [(500, 200003, torch.float32), (1100, 200003, torch.float32), (600, 2 ** 19 - 1, torch.bfloat16)])
def test_many_long_rows(T, V, dtype):
    """Long rows in CTAs of few warps, two of them a row or one; some rows in order, equal or masked."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + V)
    x = torch.randn((T, V), generator=g, device="cuda").to(dtype)
    x[3] = torch.linspace(-4, 4, V, device="cuda").to(dtype)
    x[5] = 0.5
    x[7, 100:] = -torch.inf
    x[9, :-20] = torch.finfo(dtype).min
    tokens = torch.randint(-1, V + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    some = torch.arange(0, T, 37, device="cuda")
    some = torch.cat([torch.arange(11, device="cuda"), some[some > 10], torch.tensor([T - 1], device="cuda")])
    got = msa.msa_logprobs(x, tokens, top=20)
    few = msa.msa_logprobs(x[some].contiguous(), tokens[some].contiguous(), top=20)
    _check(x[some].contiguous(), tokens[some].contiguous(), 20)
    assert torch.equal(got[1][some], few[1]) and torch.equal(got[3][some], few[3])  # ranks and best
    H = np.log(V) + 1
    tol = 2 * (1 + H) * ((V / 512 + 17) * 2.0 ** -24 + 2.0 ** -20)  # both off by one such
    for a, b in ((got[0][some], few[0]), (got[2][some] / (2 * (1 + H)), few[2] / (2 * (1 + H))), (got[4][some], few[4])):
        assert torch.equal(torch.isinf(a), torch.isinf(b))
        fine = ~torch.isinf(a)
        assert not ((a - b).abs()[fine].double() > tol + 2.0 ** -21 * a[fine].abs().double()).any()
