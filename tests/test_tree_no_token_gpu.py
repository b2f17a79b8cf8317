"""Acceptance where the target has no token (-1, the best of a row of NaN) and nodes without one."""
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


@pytest.mark.parametrize("fp4", [False, True])
def test_no_token_matches_no_token(fp4):
    accept = msa.msa_tree_accept_nvfp4 if fp4 else msa.msa_tree_accept
    pool = torch.randint(0, 120, (3, 2, 2, 9216) if fp4 else (3, 2, 128, 256), dtype=torch.uint8, device="cuda")
    before = pool.clone()
    # three requests: -1 after the root; a token that stands, then -1; -1 among the drafts beside one that stands
    drafts = i32([5, -1, -1, 5, 7, -1, 5, -1, 9])
    parents = i32([-1, 0, 1, -1, 0, 1, -1, 0, 0])
    chosen = i32([-1, -1, -1, 7, -1, -1, 9, 4, 3])
    tokens, accepted, path = accept(drafts, parents, chosen, i32([0, 3, 6, 9]), i32([0, 20, 40, 60]), 3, kv=pool, block_table=i32([[0], [1], [2]]))
    assert tokens.tolist() == [[-1, -1, -1], [7, -1, -1], [9, 3, -1]]
    assert accepted.tolist() == [0, 1, 1] and path.tolist() == [[0, -1, -1], [0, 1, -1], [0, 2, -1]]
    assert torch.equal(pool[:2], before[:2])  # (of the last request row 19 becomes row 18)
    assert not torch.equal(pool[2], before[2])
