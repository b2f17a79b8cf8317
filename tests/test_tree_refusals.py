"""What the calls around tree decoding refuse, without a GPU."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_serve_refusals import _cache, _err

# 2 pi to 50 digits
TWO_PI = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def test_turns_are_exact():
    freq = [1.0, 0.0, -1.0, 1e-3, 5e-7, 2 * math.pi, 1234567.25, 4294967295.5, 2.0 ** -60, 1e-300, 5e-324, -0.3, 3.0]
    for f, got in zip(freq, msa.msa_rope_turns(freq)):
        x = Fraction(abs(f)) / TWO_PI * 2 ** 64
        want = (int(x + Fraction(1, 2)) if f >= 0 else -int(x + Fraction(1, 2))) % 2 ** 64
        assert got == want, f
    for bad in (float("nan"), float("inf"), 4294967296.0, -1e10):
        assert "out of range" in _err(msa.msa_rope_turns, [1.0, bad])
    assert msa.msa_rope_turns([]) == []


def test_rope_refusals():
    assert "at most 64" in _err(msa.MsaRope, [1.0] * 65)
    assert "axes must be" in _err(msa.MsaRope, [1.0, 2.0], axes=[0]) and "axes must be" in _err(msa.MsaRope, [1.0], axes=[8])
    assert "eps must be" in _err(msa.MsaRope, [1.0], eps=-1.0) and "eps must be" in _err(msa.MsaRope, [1.0], eps=float("nan"))
    assert "q_norm must be a tensor [128]" in _err(msa.MsaRope, [1.0], q_norm=torch.ones(64))
    assert "k_norm must be a CUDA tensor" in _err(msa.MsaRope, [1.0], k_norm=torch.ones(128))
    rope, two = msa.MsaRope([1.0, 0.5]), msa.MsaRope([1.0, 0.5], axes=[0, 1])
    c = dict(_cache(), q=torch.zeros((6, 4, 128)), rope=rope, qs=1.0)

    def run(fn=msa.msa_rope_write, **kw):
        a = dict(c, **{k: v for k, v in kw.items() if k in c})
        return _err(fn, a["rope"], a["q"], a["k"], a["v"], a["kv"], a["qs"], 1.0, 1.0, a["table"], a["cu_q"], a["cu_k"],
                    **{k: v for k, v in kw.items() if k not in c})

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    assert "CUDA" in run() and "CUDA" in run(q=None) and "CUDA" in run(qs=None)
    assert "CUDA" in run(positions=i32(6)) and "CUDA" in run(positions=i32(1, 6)) and "CUDA" in run(rope=two, positions=i32(2, 6))
    assert "rope must be" in run(rope=None)
    assert "positions must be [1, 6] or [6]" in run(positions=i32(5)) and "positions must be [2, 6]," in run(rope=two, positions=i32(6))
    assert "positions has dtype" in run(positions=i32(6).long()) and "positions must be contiguous" in run(positions=i32(6, 2)[:, 0])
    assert "q must be" in run(q=torch.zeros((6, 512))) and "q must be [6, 4, 128]" in run(q=torch.zeros((5, 4, 128)))
    assert "different dtypes" in run(q=torch.zeros((6, 4, 128), dtype=torch.float16)) and "different dtypes" in run(v=torch.zeros((6, 2, 128)).half())
    assert "contiguous" in run(q=torch.zeros((6, 4, 256))[..., ::2])
    assert "q_out has dtype" in run(q_out=torch.zeros((6, 4, 128))) and "q_out has dtype" in run(qs=None, q_out=torch.zeros((6, 4, 128), dtype=torch.uint8))
    assert "q_out must be [6, 4, 128]" in run(q_out=torch.zeros((6, 2, 128), dtype=torch.uint8))
    assert "q_out without q" in run(q=None, q_out=torch.zeros((6, 4, 128), dtype=torch.uint8))
    assert "kv must be" in run(kv=c["kv"][:, :, :64]) and "kv4 must be" in run(msa.msa_rope_write_nvfp4)
    assert "[6, 2, 128]" in run(k=torch.zeros((6, 3, 128))) and "k and v must be" in run(v=None)
    assert "block_table must be" in run(table=c["table"][:1]) and "cu_seqlens_k must be" in run(cu_k=c["cu_k"][:2])
    assert "status" in run(status=i32(2))


def test_rope_library_refusals():
    lib, P = msa.load(), ctypes.c_void_p
    a = P(4096)  # never dereferenced: every call below ends on the host
    keep = []

    def struct(pairs=2, axes=1, eps=1e-6, axis=0, norm=None):
        s = msa.MsaRopeStruct()
        s.pairs, s.axes, s.eps, s.q_norm = pairs, axes, eps, norm
        s.axis[1] = axis
        keep.append(s)
        return ctypes.addressof(s)

    def run(rope=struct(), pos=None, q=a, qt=512, qh=128, k=a, dtype=1, out=a, bf16=0, qs=1.0, kv=a, pages=4, s=1.0, table=a, width=3, cu=a, cu_k=a, B=2, T=6,
            Hq=4, H=2, status=None, fn=lib.msa_rope_write):
        return fn(rope, pos, q, qt, qh, k, 256, 128, a, 256, 128, dtype, out, bf16, qs, kv, pages, s, 1.0, table, width, cu, cu_k, B, T, Hq, H, status, None)

    for fn in (lib.msa_rope_write, lib.msa_rope_write_nvfp4):
        assert run(B=0, fn=fn) == 0 and run(T=0, q=None, fn=fn) == 0
        assert run(rope=None, fn=fn) == 6 and run(q=None, fn=fn) == 6 and run(k=None, fn=fn) == 6 and run(out=None, fn=fn) == 6 and run(kv=None, fn=fn) == 6
        assert run(table=None, fn=fn) == 6 and run(cu=None, fn=fn) == 6 and run(cu_k=None, fn=fn) == 6
        assert run(dtype=3, fn=fn) == 2
        for bad in (dict(pairs=65), dict(pairs=-1), dict(axes=0), dict(axes=9), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=1e39), dict(axis=1)):
            assert run(rope=struct(**bad), fn=fn) == 1
        assert run(rope=struct(axes=2, axis=1), T=0, fn=fn) == 0
        for bad in (dict(T=-1), dict(B=-1), dict(H=0), dict(H=128), dict(Hq=-1), dict(Hq=127 * 128 + 1), dict(T=2 ** 31), dict(pages=-1), dict(width=-1),
                    dict(qt=-8), dict(width=2 ** 24 + 1)):
            assert run(fn=fn, **bad) == 1
        for s in (0.0, -1.0, float("nan"), float("inf")):
            assert run(s=s, fn=fn) == 1 and run(qs=s, fn=fn) == 1 and run(qs=s, bf16=1, T=0, fn=fn) == 0 and run(qs=s, Hq=0, T=0, fn=fn) == 0
        assert run(qt=516, fn=fn) == 3 and run(qh=129, fn=fn) == 3 and run(q=P(4104), fn=fn) == 3 and run(out=P(4104), fn=fn) == 3
        assert run(pos=P(4097), fn=fn) == 3 and run(rope=struct(norm=4097), fn=fn) == 3 and run(status=P(4098), fn=fn) == 3
    assert run(s=1e38, fn=lib.msa_rope_write_nvfp4, T=0) == 1 and run(s=1e38, T=0) == 0
    turns = (ctypes.c_uint64 * 1)()
    assert lib.msa_rope_turns(None, 1, turns) == 6 and lib.msa_rope_turns(None, -1, turns) == 1 and lib.msa_rope_turns(None, 0, None) == 0


@pytest.mark.parametrize("at,bad", [(0, True), (600, True), (1 << 20, False)])
def test_rope_refuses_an_output_over_its_inputs(at, bad):
    # checked behind the device's check, so by the bounds alone here
    from block_sparse_attention_prefill_gb300.tree import _reach

    room = torch.zeros((1 << 21,), dtype=torch.uint8)
    q = room[:6 * 1024].view(6, 8, 128)[:, :4]
    out = room[at:at + 6 * 512].view(6, 4, 128)
    (lo, hi), (a, b) = _reach(out), _reach(q)
    assert (a < hi and lo < b) is bad


i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731


def test_mask_refusals():
    run = lambda p=i32(6), q=i32(3), k=i32(3), n=6, **kw: _err(msa.msa_tree_mask, p, q, k, n, **kw)  # noqa: E731
    assert "CUDA" in run() and "CUDA" in run(mask=i32(6, 1), positions=i32(6))
    assert "parents has dtype" in run(p=i32(6).long()) and "parents must be [T]" in run(p=i32(3, 2)) and "parents must be contiguous" in run(p=i32(6, 2)[:, 0])
    assert "cu_seqlens_k must be" in run(k=i32(2)) and "at least one" in run(q=i32(0)) and "parents is required" in run(p=None)
    assert "mask must be [6, 2]" in run(n=33, mask=i32(6, 1)) and "positions must be" in run(positions=i32(5))
    assert "0 .. 256" in run(n=257) and "0 .. 256" in run(n=-1)
    assert "status" in run(status=i32(2))


def test_tree_attention_refusals():
    a = {"q": torch.zeros((6, 4, 128), dtype=torch.uint8), "kv": torch.zeros((4, 2, 128, 256), dtype=torch.uint8), "table": i32(2, 3), "cu_q": i32(3),
         "cu_k": i32(3), "mask": i32(6, 1), "prefix": 1, "max_q": 6, "max_k": 300}

    def run(**kw):
        c = dict(a, **{k: v for k, v in kw.items() if k in a})
        return _err(msa.msa_tree_attention, c["q"], c["kv"], 1.0, 1.0, 1.0, 0.1, c["table"], c["cu_q"], c["cu_k"], c["mask"], c["prefix"], c["max_q"],
                    c["max_k"], **{k: v for k, v in kw.items() if k not in a})

    assert "CUDA" in run() and "CUDA" in run(mask=i32(6, 3))
    assert "mask must be [6, 2 or more]" in run(max_q=33) and "mask must be [6, 1 or more]" in run(mask=i32(5, 1)) and "mask must be" in run(mask=i32(6))
    assert "mask has dtype" in run(mask=i32(6, 1).long()) and "mask must be contiguous" in run(mask=i32(6, 2)[:, :1]) and "mask is required" in run(mask=None)
    assert "0 .. 256" in run(max_q=257) and "mask must be [T" in run(q=None)
    assert "q has dtype" in run(q=a["q"].to(torch.bfloat16)) and "workspace too small" in run(workspace=torch.zeros(100, dtype=torch.uint8))
    assert "out of range" in run(prefix=3) and "unsupported" in run(q=torch.zeros((6, 3, 128), dtype=torch.uint8))


def test_accept_refusals():
    kv, kv4 = torch.zeros((4, 2, 128, 256), dtype=torch.uint8), torch.zeros((4, 2, 2, 9216), dtype=torch.uint8)

    def run(d=i32(6), p=i32(6), c=i32(6), q=i32(3), k=i32(3), n=6, fn=msa.msa_tree_accept, **kw):
        return _err(fn, d, p, c, q, k, n, **kw)

    table = i32(2, 3)
    assert "CUDA" in run() and "CUDA" in run(kv=kv, block_table=table) and "CUDA" in run(kv=[kv, kv.clone()], block_table=table)
    assert "CUDA" in run(kv=torch.stack([kv, kv]), block_table=table) and "CUDA" in run(kv=kv4, block_table=table, fn=msa.msa_tree_accept_nvfp4)
    assert "draft_tokens has dtype" in run(d=i32(6).long()) and "parents must be [6]" in run(p=i32(5)) and "chosen must be [6]" in run(c=i32(5))
    assert "cu_seqlens_k must be" in run(k=i32(2)) and "0 .. 256" in run(n=300) and "chosen is required" in run(c=None)
    assert "tokens must be [2, 6]" in run(tokens=i32(2, 5)) and "accepted must be" in run(accepted=i32(3)) and "path must be" in run(path=i32(2, 7))
    assert "kv must be" in run(kv=kv[:, :, :64], block_table=table) and "kv must be" in run(kv=kv4, block_table=table)
    assert "kv4 must be" in run(kv=kv, block_table=table, fn=msa.msa_tree_accept_nvfp4)
    assert "pools differ" in run(kv=[kv, kv[:3].contiguous()], block_table=table)
    assert "block_table is required" in run(kv=kv) and "block_table must be" in run(kv=kv, block_table=i32(3, 3))
    assert "at most 128 layers" in run(kv=[kv] * 129, block_table=table)


def test_logprobs_refusals():
    x, t = torch.zeros((4, 50)), i32(4)
    run = lambda x=x, t=t, **kw: _err(msa.msa_logprobs, x, t, **kw)  # noqa: E731
    assert "CUDA" in run() and "CUDA" in run(t=None) and "CUDA" in run(x=torch.zeros((4, 80))[:, :50])
    assert "top must be 0 .. 32" in run(top=33) and "top must be" in run(top=-1)
    assert "logits must be [T, V]" in run(x=torch.zeros((2, 2, 50))) and "logits has dtype" in run(x=x.double()) and "rows must be contiguous" in run(x=x.T)
    assert "tokens must be [4]" in run(t=i32(5)) and "tokens has dtype" in run(t=t.long())
    assert "logprobs and ranks need tokens" in run(t=None, ranks=i32(4))
    assert "logprobs must be [4]" in run(logprobs=torch.zeros(5)) and "top_tokens must be [4, 2]" in run(top=2, top_tokens=i32(4, 3))
    assert "entropy has dtype" in run(entropy=torch.zeros(4, dtype=torch.float64))


def test_outputs_that_share_memory():
    from block_sparse_attention_prefill_gb300.tree import _apart

    room = torch.zeros(100)
    for a, b, bad in ((room[:10], room[9:20], True), (room[:10], room[10:20], False), (room[:0], room, False), (room[5:95].view(9, 10)[:, :2], room[90:], False),
                      (room[5:95].view(9, 10)[:, :2], room[86:], True)):
        for outs, inputs in (({"a": a, "b": b}, {}), ({"a": a}, {"b": b, "c": None}), ({"b": b, "d": None}, {"a": a})):
            if bad:
                assert "must not share memory" in _err(_apart, outs, inputs)
            else:
                _apart(outs, inputs)


def test_tree_library_refusals():
    lib, P = msa.load(), ctypes.c_void_p
    a = P(4096)

    def mask(p=a, q=a, k=a, B=2, T=6, n=6, m=a, pos=a, status=None):
        return lib.msa_tree_mask(p, q, k, B, T, n, m, pos, status, None)

    assert mask(B=0) == 0 and mask(T=0, p=None) == 0
    assert mask(p=None) == 6 and mask(q=None) == 6 and mask(k=None) == 6
    assert mask(n=257) == 1 and mask(n=-1) == 1 and mask(B=-1) == 1 and mask(T=-1) == 1 and mask(T=2 ** 31) == 1
    assert mask(p=P(4098)) == 3 and mask(m=P(4097)) == 3 and mask(pos=P(4097)) == 3 and mask(status=P(4097)) == 3

    def attend(q=a, m=a, words=1, n=6, T=6, s=1.0, ws=a, size=1 << 40, width=3, Hq=4, out=a):
        return lib.msa_tree_attention(q, a, 4, s, 1.0, 1.0, 0.1, a, width, a, a, m, words, 2, T, Hq, 2, 1, n, 300, ws, size, out, None, None, None)

    assert attend(T=0) == 0 and attend(m=None) == 6 and attend(q=None) == 6 and attend(out=None) == 6
    assert attend(words=0) == 1 and attend(n=33) == 1 and attend(n=257, words=20) == 1 and attend(width=2) == 1 and attend(s=0.0) == 1
    assert attend(Hq=3) == 2 and attend(ws=None) == 4 and attend(size=100) == 4 and attend(m=P(4098)) == 3 and attend(q=P(4104)) == 3

    def accept(d=a, p=a, c=a, q=a, B=2, T=6, n=6, pools=(1 << 20, 2 << 20), pages=4, H=2, table=a, width=3, tokens=a, accepted=a, path=None, status=None,
               fn=lib.msa_tree_accept, layers=None):
        at = (ctypes.c_uint64 * max(len(pools), 1))(*pools)
        return fn(d, p, c, q, a, B, T, n, ctypes.addressof(at), len(pools) if layers is None else layers, pages, H, table, width, tokens, accepted, path,
                  status, None)

    for fn in (lib.msa_tree_accept, lib.msa_tree_accept_nvfp4):
        assert accept(B=0, fn=fn) == 0
        assert accept(d=None, fn=fn) == 6 and accept(p=None, fn=fn) == 6 and accept(c=None, fn=fn) == 6 and accept(q=None, fn=fn) == 6
        assert accept(tokens=None, fn=fn) == 6 and accept(accepted=None, fn=fn) == 6 and accept(table=None, fn=fn) == 6 and accept(pools=(0, 4096), fn=fn) == 6
        for bad in (dict(n=257), dict(n=-1), dict(B=-1), dict(T=-1), dict(H=0), dict(H=128), dict(pages=-1), dict(width=-1), dict(layers=129), dict(layers=-1)):
            assert accept(fn=fn, **bad) == 1
        # pools that share memory: one twice, one that begins in another, in any order
        assert accept(pools=(1 << 20, 1 << 20), fn=fn) == 1 and accept(pools=(2 << 20, 9 << 20, (2 << 20) + 64 * 1024), fn=fn) == 1
        assert accept(pools=((1 << 20) + 8, 9 << 20), fn=fn) == 3 and accept(path=P(4097), fn=fn) == 3 and accept(status=P(4097), fn=fn) == 3
    edge = 4 * 2 * 32768  # two pools end to end are apart
    assert accept(pools=(1 << 20, (1 << 20) + edge), status=P(4097)) == 3 and accept(pools=(1 << 20, (1 << 20) + edge - 16)) == 1

    def logprobs(x=a, row=50, dtype=0, t=a, T=4, V=50, top=2, lp=a, r=a, e=a, tt=a, tl=a):
        return lib.msa_logprobs(x, row, dtype, t, T, V, top, lp, r, e, tt, tl, None)

    assert logprobs(T=0, x=None) == 0 and logprobs(dtype=3) == 2
    assert logprobs(x=None) == 6 and logprobs(t=None) == 6 and logprobs(tt=None) == 6 and logprobs(tl=None) == 6 and logprobs(t=None, lp=None) == 6
    for bad in (dict(T=-1), dict(T=2 ** 31), dict(V=0), dict(V=2 ** 19), dict(row=-1), dict(top=33), dict(top=-1)):
        assert logprobs(**bad) == 1
    assert logprobs(x=P(4098)) == 3 and logprobs(x=P(4097), dtype=1) == 3 and logprobs(t=P(4097)) == 3 and logprobs(e=P(4097)) == 3


def test_tensors_of_another_device_are_refused(monkeypatch):
    class Other(torch.Tensor):
        def get_device(self):
            return 3

    on = lambda t: t.as_subclass(Other)  # noqa: E731
    z = lambda *s: on(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    u8 = lambda *s: on(torch.zeros(s, dtype=torch.uint8))  # noqa: E731
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    kv = u8(4, 2, 128, 256)
    x = on(torch.zeros((6, 2, 128)))
    for call in (lambda: msa.msa_rope_write(msa.MsaRope([1.0]), x, x, x, kv, 1.0, 1.0, 1.0, z(2, 3), z(3), z(3)),
                 lambda: msa.msa_tree_mask(z(6), z(3), z(3), 6),
                 lambda: msa.msa_tree_attention(u8(6, 4, 128), kv, 1.0, 1.0, 1.0, 0.1, z(2, 3), z(3), z(3), z(6, 1), 1, 6, 300),
                 lambda: msa.msa_tree_accept(z(6), z(6), z(6), z(3), z(3), 6, kv=[kv], block_table=z(2, 3)),
                 lambda: msa.msa_logprobs(on(torch.zeros((6, 50))), z(6), top=2)):
        assert "the current device is cuda:0" in _err(call)
