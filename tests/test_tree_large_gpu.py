"""Pools, projections and lengths whose places pass 32 bits, against the same
call on small ones."""
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


@pytest.mark.parametrize("fp4", [False, True])
def test_pools_beyond_4_gb(fp4):
    """Rows written and moved in the last pages of a pool of 5 GB are those of a pool of four pages."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    pages = 140000 if fp4 else 80000
    shape = (2, 2, 9216) if fp4 else (2, 128, 256)
    big, small = torch.zeros((pages,) + shape, dtype=torch.uint8, device="cuda"), torch.zeros((4,) + shape, dtype=torch.uint8, device="cuda")
    x = torch.randn((20, 6, 128), generator=g, device="cuda").bfloat16()
    cu_q, cu_k = i32([0, 20]), i32([0, 140])
    write, accept = (msa.msa_rope_write_nvfp4, msa.msa_tree_accept_nvfp4) if fp4 else (msa.msa_rope_write, msa.msa_tree_accept)
    rope = msa.MsaRope([1.0 / (j + 1) for j in range(48)])
    parents, drafts = i32([-1] + [max(0, i - 2) for i in range(1, 20)]), torch.arange(20, device="cuda", dtype=torch.int32)
    chosen = drafts + 2  # every second node
    chosen[0] = 2
    for pool, table in ((big, i32([[pages - 1, pages - 3]])), (small, i32([[3, 1]]))):
        write(rope, x[:, :2], x[:, 2:4], x[:, 4:], pool, 0.0131, 0.0127, 0.0149, table, cu_q, cu_k)
        tokens, accepted, path = accept(drafts, parents, chosen, cu_q, cu_k, 20, kv=pool, block_table=table)
        assert accepted.item() == 9 and path[0, :10].tolist() == list(range(0, 20, 2))
    assert torch.equal(big[-4:], small)
    assert not big[:-4].any()


def test_projections_beyond_2_31_values():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    T, hq, hkv = 270000, 60, 2
    x = torch.zeros((T, hq + 2 * hkv, 128), dtype=torch.bfloat16, device="cuda")
    last = torch.randn((50, hq + 2 * hkv, 128), generator=g, device="cuda").bfloat16()
    x[-50:] = last
    pages = -(-T // 128)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    kv = torch.zeros((pages, hkv, 128, 256), dtype=torch.uint8, device="cuda")
    rope = msa.MsaRope([1.0 / (j + 1) for j in range(64)])
    q = msa.msa_rope_write(rope, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kv, 0.0131, 0.0127, 0.0149, table, i32([0, T]), i32([0, T]))
    other = kv.clone()
    want = msa.msa_rope_write(rope, last[:, :hq], last[:, hq:hq + hkv], last[:, hq + hkv:], other, 0.0131, 0.0127, 0.0149, table, i32([0, 50]), i32([0, T]))
    assert torch.equal(q[-50:].view(torch.uint8), want.view(torch.uint8)) and torch.equal(kv, other)
