"""Which stream's memory a call's outputs and workspace come from when it is
given another stream than the current one: that stream's, since a free block
of the current one's may still be read or written by what is queued there."""
import contextlib
import types

import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from block_sparse_attention_prefill_gb300 import serve


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def streams(monkeypatch):
    """Streams without a GPU: the current one's handle is the list's last, and
    tensors remember the stream they were made on and those recorded."""
    now = [_Stream(5)]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    def empty(shape, dtype, device):
        t = types.SimpleNamespace(made_on=now[-1].cuda_stream, used_on=[], device=device)
        t.record_stream = lambda s: t.used_on.append(s.cuda_stream)
        return t

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _Stream(handle or 999))  # (of 0: a new one)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: now[-1].cuda_stream, raising=False)
    return now


def test_outputs_come_from_the_streams_memory(streams):
    for handle in (77, 0):
        t = serve._new((4,), torch.int32, 0, handle)
        assert t.made_on == handle and t.used_on == [5]
    t = serve._new((4,), torch.int32, 0, 5)
    assert t.made_on == 5 and t.used_on == []
    assert streams[-1].cuda_stream == 5


def _verify(V=64, B=300):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    target = torch.softmax(torch.randn((B, 3, V), generator=g, device="cuda"), -1)
    drafts = torch.randint(0, V, (B, 2), generator=g, device="cuda", dtype=torch.int32)
    return target, drafts, torch.rand((B, 3), generator=g, device="cuda")


@pytest.mark.gpu
def test_blocks_freed_on_the_current_stream_are_not_taken():
    target, drafts, u = _verify()
    want = msa.msa_verify(target, drafts, u)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, free on the current stream
    held = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((300, 3), (300,)) for _ in range(40)]
    free = {t.data_ptr() for t in held}
    del held
    for stream in (side, side.cuda_stream):
        got = msa.msa_verify(target, drafts, u, stream=stream)
        assert not free & {t.data_ptr() for t in got}
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the default stream by its handle, 0, from a block under another one
    with torch.cuda.stream(side):
        held = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((300, 3), (300,)) for _ in range(40)]
        free = {t.data_ptr() for t in held}
        del held
        got = msa.msa_verify(target, drafts, u, stream=0)
        assert not free & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_older_calls_workspace_comes_from_the_streams_memory(streams):
    t = msa._workspace(100, "cuda:0", None, 77)
    assert t.made_on == 77 and t.used_on == [5]
    t = msa._workspace(100, "cuda:0", None, None)
    assert t.made_on == 5 and t.used_on == []


@pytest.mark.gpu
def test_older_calls_take_no_blocks_freed_on_the_current_stream():
    import workloads
    w = workloads.make_batch("streams", [160, 48], [2600, 700], 16, 2, seed=0).to("cuda:0")
    want = msa.run_workload(w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    T = w.q.shape[0]
    part_o, part_lse = torch.randn((50, 3, 128), device="cuda"), torch.randn((50, 3), device="cuda")
    merged = msa.msa_combine(part_o, part_lse)
    sizes = [T * 16 * 128 * 2, T * 16 * 4, want[2].workspace.numel(), msa.prefill_workspace_bytes(T, 16), 50 * 128 * 2, 50 * 4]
    torch.cuda.synchronize()
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]
    del held
    got = msa.run_workload(w, stream=side)
    again = msa.msa_combine(part_o, part_lse, stream=side)
    for t in (got[0], got[1], got[2].workspace, *again):
        assert not any(a < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < b for a, b in spans)
    side.synchronize()
    assert got[2].status() == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(a, b) for a, b in zip(again, merged))


def test_a_workspace_size_is_kept_for_the_current_device_only(monkeypatch):
    # the library gives the current device's size: tensors of another device
    # have to be refused, and nothing be kept under theirs
    class Other(torch.Tensor):
        def get_device(self):
            return 3

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32).as_subclass(Other)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8).as_subclass(Other)  # noqa: E731
    asked = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(serve, "_attention_bytes", lambda *a: asked.append(a) or 1 << 20)
    with pytest.raises(msa.MsaError, match="current device is cuda:0"):
        msa.msa_prefix_attention(u8(6, 4, 128), u8(4, 2, 128, 256), 1.0, 1.0, 1.0, 0.1, i32(2, 3), i32(3), i32(3), 1, 6, 300)
    assert not asked
