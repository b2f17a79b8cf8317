"""The tree calls on another stream than the current one: outputs from that
stream's memory, not from blocks that are free on the current one's; and two
calls at once, on two streams, that know nothing of each other."""
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731


def _calls():
    """The calls, as functions of keyword arguments, with the bytes of their outputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    B, n, hq, hkv = 9, 20, 8, 2
    T = B * n
    cu_q, cu_k = i32([i * n for i in range(B + 1)]), i32([i * 300 for i in range(B + 1)])
    table = torch.randperm(B * 3, generator=g, device="cuda").to(torch.int32).view(B, 3)
    parents = i32(([-1] + [i // 2 for i in range(n - 1)]) * B)
    drafts, chosen = (torch.randint(0, 3, (T,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2))
    x = rand(T, hq + 2 * hkv, 128).bfloat16()
    kv = (rand(B * 3, hkv, 128, 256) / 0.013).to(torch.float8_e4m3fn)
    q8 = (rand(T, hq, 128) / 0.013).to(torch.float8_e4m3fn)
    rope = msa.MsaRope([1.0 / (j + 1) for j in range(32)])
    mask, _ = msa.msa_tree_mask(parents, cu_q, cu_k, n)
    logits = rand(T, 700)
    pools = [kv.clone(), kv.clone()]
    return {
        "rope": lambda **k: msa.msa_rope_write(rope, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kv.clone(), 0.0131, 0.0127, 0.0149, table, cu_q, cu_k, **k),
        "mask": lambda **k: msa.msa_tree_mask(parents, cu_q, cu_k, n, **k),
        "attend": lambda **k: msa.msa_tree_attention(q8, kv, 0.0131, 0.0127, 0.0149, 0.09, table, cu_q, cu_k, mask, 0, n, 300, **k),
        "accept": lambda **k: msa.msa_tree_accept(drafts, parents, chosen, cu_q, cu_k, n, kv=[p.clone() for p in pools] if k.get("stream") is None else None,
                                                  block_table=table, **k),
        "logprobs": lambda **k: msa.msa_logprobs(logits, drafts, top=5, **k),
    }


def _bytes(out):
    return [t.contiguous().view(torch.uint8) for t in (out if isinstance(out, tuple) else (out,))]


@pytest.mark.parametrize("name", ["rope", "mask", "attend", "accept", "logprobs"])
def test_blocks_freed_on_the_current_stream_are_not_taken(name):
    call = _calls()[name]
    want = _bytes(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    held = [torch.empty(t.numel(), dtype=torch.uint8, device="cuda") for t in want for _ in range(40)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]
    torch.cuda.synchronize()
    del held
    for stream in (side, side.cuda_stream):
        got = _bytes(call(stream=stream))
        side.synchronize()
        for t, v in zip(got, want):
            assert not any(a < t.data_ptr() + t.numel() and t.data_ptr() < b for a, b in spans)
            assert torch.equal(t, v)


def test_two_streams_at_once():
    calls = _calls()
    want = {k: _bytes(f()) for k, f in calls.items()}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append({k: calls[k]() for k in ("mask", "attend", "logprobs")})
        torch.cuda.synchronize()
        for g in got:
            for k, out in g.items():
                assert all(torch.equal(a, b) for a, b in zip(_bytes(out), want[k]))
