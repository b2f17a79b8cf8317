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

    def struct(pairs=2, axes=1, eps=1e-6, axis=0, norm=None):
        s = msa.MsaRopeStruct()
        s.pairs, s.axes, s.eps, s.q_norm = pairs, axes, eps, norm
        s.axis[1] = axis
        return ctypes.byref(s)

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
