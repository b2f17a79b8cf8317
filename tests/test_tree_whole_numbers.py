"""Sizes of the tree calls have to be whole numbers: a fraction is refused, not cut off."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_serve_refusals import _err

i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731


@pytest.mark.parametrize("bad", [2.5, float("nan"), float("inf"), "6", None])
def test_fractions_are_refused(bad):
    assert "max_seqlen_q must be a whole number" in _err(msa.msa_tree_mask, i32(6), i32(3), i32(3), bad)
    assert "max_seqlen_q must be a whole number" in _err(msa.msa_tree_accept, i32(6), i32(6), i32(6), i32(3), i32(3), bad)
    kv, q = torch.zeros((4, 2, 128, 256), dtype=torch.uint8), torch.zeros((6, 4, 128), dtype=torch.uint8)
    assert "max_seqlen_q must be a whole number" in _err(msa.msa_tree_attention, q, kv, 1.0, 1.0, 1.0, 0.1, i32(2, 3), i32(3), i32(3), i32(6, 1), 0, bad, 300)
    assert "top must be a whole number" in _err(msa.msa_logprobs, torch.zeros((4, 50)), i32(4), top=bad)
    assert "an axis must be a whole number" in _err(msa.MsaRope, [1.0, 2.0], axes=[0, bad])


def test_other_whole_numbers_are_taken():
    for n in (np.int64(6), np.int32(6), 6.0, np.float32(6), torch.tensor(6), torch.tensor(6.0)):
        assert "CUDA" in _err(msa.msa_tree_mask, i32(6), i32(3), i32(3), n)
        assert "CUDA" in _err(msa.msa_logprobs, torch.zeros((4, 50)), i32(4), top=n)
    assert msa.MsaRope([1.0, 2.0], axes=torch.tensor([0, 2])).axes == 3
