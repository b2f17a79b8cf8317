"""Log probabilities of logits of any finite size: rows masked with finite numbers
(-1e9, -1e10, -1e30, ...) in part or whole, and rows that lie far from 0.

Tolerance of the sums, from the roundings, for the smallest CTAs that take a row
(128 threads with two sums each, then their merge): n = ceil(V / 256) + 24
additions in the longest chain.  A term e^d is off by less than 2^-21 of itself
plus 2^-23 |d| (the difference d, its product with log2 e and the power), and
p |d| < 1 for any term, so l and s are off by less than (n 2^-24 + 2^-20) of
l (1 + the mean |d|), which is log V + 1 at most.  A log probability's own
difference and last roundings add 2^-22 of it."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_logprobs_gpu import _reference

pytestmark = pytest.mark.gpu

FILLS = [-6e4, -9e5, -1e6, -1.1e6, -1e9, -1e10, -1e12, -1e20, -1e30, -1.9e38, -2.1e38, 1e9, 1e10, 1e20, 1.9e38, 2.1e38]


def _check(x, tokens, top):
    T, V = x.shape
    logprob, rank, entropy, best, value = msa.msa_logprobs(x, tokens, top=top)
    a, b, c, d, e = _reference(x.double(), tokens, top)
    assert torch.equal(rank.long(), b) and torch.equal(d, best.long())
    fine = ~(x == torch.inf).any(-1)  # (the others are NaN as documented)
    assert torch.isnan(logprob[~fine]).all() and torch.isnan(entropy[~fine]).all() and torch.isnan(value[~fine]).all()
    logprob, entropy, value, a, c, e = (t[fine] for t in (logprob, entropy, value, a, c, e))
    H = np.log(V) + 1
    tol = (1 + H) * ((V / 256 + 25) * 2.0 ** -24 + 2.0 ** -20)
    for got, want in ((logprob, a), (value, e)):
        assert not torch.isnan(got).any() and torch.equal(torch.isinf(got), torch.isinf(want.float()))
        fine = ~torch.isinf(got)
        err = (got.double() - want).abs()[fine] - 2.0 ** -22 * want.abs()[fine]
        assert not (err > tol).any()
    err = (entropy.double() - c).abs()
    assert not (err > 2 * tol * (1 + H)).any()


# rows of one CTA of 16, 8 or 4 warps, and of clusters
SIZES = [(5, 900), (5, 40000), (40, 131072), (5, 200003), (700, 20000)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V", SIZES)
def test_rows_masked_with_a_number(T, V, dtype):
    """Wholly, but for ten values, in their first or second half, every other value."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    some = 3 * torch.randn((T, V), generator=g, device="cuda")
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    at = torch.arange(V, device="cuda")
    kept = torch.zeros((5, V), dtype=torch.bool, device="cuda")
    kept[1, torch.randperm(V, generator=g, device="cuda")[:10]] = True
    kept[2], kept[3], kept[4] = at >= V // 2, at < V // 2, at % 2 == 0
    kept = kept[torch.arange(T, device="cuda") % 5]
    tokens[1] = int(kept[1].nonzero()[3])
    for fill in FILLS:
        _check(torch.where(kept, some, fill).to(dtype), tokens, 12)


@pytest.mark.parametrize("T,V", SIZES)
def test_rows_far_from_zero(T, V):
    """Rows around a far number, their values a few apart and on both sides of it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V + 1)
    near = 3 * torch.randn((T, V), generator=g, device="cuda")
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    for far in (6.5e4, 9.9999e5, 1e6, 1.0001e6, 4e6, 1.6e7, 1e9):
        for x in (near + far, near - far):
            _check(x, tokens, 5)
    for size in (1e5, 1e6, 3e6, 1e10, 1e30, 1e37, 5e37):  # (the last: with infinities)
        _check(near * size, tokens, 5)


def test_half_rows_far_from_zero():
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = (torch.randn((4, 50001), generator=g, device="cuda") * 2 + 6e4).half()
    tokens = torch.arange(4, dtype=torch.int32, device="cuda")
    _check(x, tokens, 32)
    _check(-x, tokens, 32)
