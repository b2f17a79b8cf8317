"""An MsaRope made on one stream and used on another at once."""
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def test_weights_are_there_for_every_stream():
    x = torch.randn((40, 4, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.linspace(0.5, 2, 128, device="cuda").bfloat16()
    table, cu = i32([[0]]), i32([0, 40])
    kv = torch.zeros((1, 1, 128, 256), dtype=torch.uint8, device="cuda")
    freq = [1.0 / (j + 1) for j in range(64)]
    call = lambda rope: msa.msa_rope_write(rope, x[:, :2], x[:, 2:3], x[:, 3:], kv, 0.0131, 0.0127, 0.0149, table, cu, cu)  # noqa: E731
    want = call(msa.MsaRope(freq, q_norm=w, k_norm=w)).view(torch.uint8)
    torch.cuda.synchronize()
    late, other = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(late):
            torch.cuda._sleep(200_000_000)  # a tenth of a second of work ahead of the copies
            rope = msa.MsaRope(freq, q_norm=w, k_norm=w)
            assert late.query()
        with torch.cuda.stream(other):
            got = call(rope)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.uint8), want)


def test_made_while_captured():
    x = torch.randn((40, 4, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.ones(128, device="cuda")
    kv = torch.zeros((1, 1, 128, 256), dtype=torch.uint8, device="cuda")
    table, cu = i32([[0]]), i32([0, 40])
    call = lambda rope: msa.msa_rope_write(rope, x[:, :2], x[:, 2:3], x[:, 3:], kv, 0.0131, 0.0127, 0.0149, table, cu, cu)  # noqa: E731
    want = call(msa.MsaRope([0.5], q_norm=w)).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope = msa.MsaRope([0.5], q_norm=w)
        got = call(rope)
    graph.replay()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
