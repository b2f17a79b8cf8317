"""What the cache, attention and verification calls refuse, without a GPU:
the binding's checks of shapes, types, strides and devices run before the
library sees a pointer, and the library's own before anything is launched."""
import ctypes

import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa


def _err(fn, *args, **kw):
    with pytest.raises(msa.MsaError) as e:
        fn(*args, **kw)
    return str(e.value)


def _cache(T=6, H=2, B=2, pages=4):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return {"k": torch.zeros((T, H, 128)), "v": torch.zeros((T, H, 128)),
            "kv": torch.zeros((pages, H, 128, 256), dtype=torch.uint8), "table": i32(B, 3), "cu_q": i32(B + 1), "cu_k": i32(B + 1)}


def _write(c, fn=msa.msa_kv_write, **kw):
    return _err(fn, c["k"], c["v"], c["kv"], 1.0, 1.0, c["table"], c["cu_q"], c["cu_k"], **kw)


def test_write_refusals():
    c = _cache()
    assert "CUDA" in _write(c)
    assert "[6, 2, 128]" in _write(dict(c, v=torch.zeros((6, 3, 128))))
    assert "[6, 2, 128]" in _write(dict(c, v=torch.zeros((5, 2, 128))))
    assert "different dtypes" in _write(dict(c, v=torch.zeros((6, 2, 128), dtype=torch.float16)))
    assert "dtype" in _write(dict(c, k=c["k"].double()))
    assert "contiguous" in _write(dict(c, k=torch.zeros((6, 2, 256))[..., ::2]))
    assert "kv must be" in _write(dict(c, kv=c["kv"][:, :, :64]))
    assert "kv must be contiguous" in _write(dict(c, kv=torch.zeros((4, 3, 128, 256), dtype=torch.uint8)[:, :2]))
    assert "kv4 must be" in _write(c, msa.msa_kv_write_nvfp4)
    assert "block_table must be" in _write(dict(c, table=c["table"][:1]))
    assert "block_table must be" in _write(dict(c, table=c["table"][0]))
    assert "block_table has dtype" in _write(dict(c, table=c["table"].long()))
    assert "cu_seqlens_k must be" in _write(dict(c, cu_k=c["cu_k"][:2]))
    assert "at least one" in _write(dict(c, cu_q=c["cu_q"][:0]))
    assert "status" in _write(c, status=torch.zeros(2, dtype=torch.int32))
    assert "k and v must be" in _write(dict(c, k=None))


def test_read_refusals():
    c = _cache()
    run = lambda fn=msa.msa_kv_read, total=6, **kw: _err(fn, kw.pop("kv", c["kv"]), 1.0, 1.0, c["table"], c["cu_q"], total, **kw)  # noqa: E731
    assert "CUDA" in run()
    assert "starts must be" in run(starts=torch.zeros(3, dtype=torch.int32))
    assert "kv has dtype" in run(kv=c["kv"].to(torch.int8))


def test_verify_refusals():
    t, d, x, u = torch.zeros((2, 4, 50)), torch.zeros((2, 3, 50)), torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 4))
    assert "CUDA" in _err(msa.msa_verify, t, x, u, d)
    assert "CUDA" in _err(msa.msa_verify_greedy, t, x)
    assert "target must be" in _err(msa.msa_verify, t[0], x, u, d)
    assert "at least one row" in _err(msa.msa_verify_greedy, t[:, :0], x)
    assert "rows must be contiguous" in _err(msa.msa_verify, t.transpose(1, 2), x, u, d)
    assert "draft_tokens must be" in _err(msa.msa_verify, t, x[:, :2], u, d)
    assert "draft_tokens has dtype" in _err(msa.msa_verify, t, x.long(), u, d)
    assert "uniforms must be" in _err(msa.msa_verify, t, x, u[:, :3], d)
    assert "uniforms has dtype" in _err(msa.msa_verify, t, x, u.double(), d)
    assert "draft_probs must be" in _err(msa.msa_verify, t, x, u, t)
    assert "draft_probs has dtype" in _err(msa.msa_verify, t, x, u, d.half())
    assert "num_drafts must be" in _err(msa.msa_verify, t, x, u, d, torch.zeros(3, dtype=torch.int32))


def test_library_refusals():
    lib, P = msa.load(), ctypes.c_void_p
    a = P(4096)  # never dereferenced: every call below ends on the host

    def write(k=a, kt=256, kh=128, dtype=1, kv=a, pages=4, s=1.0, table=a, width=3, cu_q=a, cu_k=a, B=2, T=6, H=2, status=None, fn=lib.msa_kv_write):
        return fn(k, kt, kh, a, 256, 128, dtype, kv, pages, s, 1.0, table, width, cu_q, cu_k, B, T, H, status, None)

    for fn in (lib.msa_kv_write, lib.msa_kv_write_nvfp4):
        assert write(B=0, fn=fn) == 0 and write(T=0, k=None, fn=fn) == 0
        assert write(k=None, fn=fn) == 6 and write(kv=None, fn=fn) == 6 and write(table=None, fn=fn) == 6
        assert write(cu_q=None, fn=fn) == 6 and write(cu_k=None, fn=fn) == 6
        assert write(dtype=3, fn=fn) == 2
        assert write(T=-1, fn=fn) == 1 and write(B=-1, fn=fn) == 1 and write(H=0, fn=fn) == 1 and write(H=128, fn=fn) == 1
        assert write(T=2 ** 31, fn=fn) == 1 and write(pages=-1, fn=fn) == 1 and write(width=-1, fn=fn) == 1
        for s in (0.0, -1.0, float("nan"), float("inf")):
            assert write(s=s, fn=fn) == 1
        assert write(kt=-256, fn=fn) == 1
        assert write(kt=260, fn=fn) == 3 and write(kh=129, fn=fn) == 3 and write(k=P(4104), fn=fn) == 3
        assert write(kv=P(4104), fn=fn) == 3 and write(cu_q=P(4098), fn=fn) == 3 and write(status=P(4098), fn=fn) == 3

    def read(kv=a, cu=a, starts=None, k=a, dtype=0, T=6, s=1.0, fn=lib.msa_kv_read):
        return fn(kv, 4, s, 1.0, a, 3, cu, starts, 2, T, 2, k, 256, 128, a, 256, 128, dtype, None, None)

    for fn in (lib.msa_kv_read, lib.msa_kv_read_nvfp4):
        assert read(kv=None, fn=fn) == 6 and read(cu=None, fn=fn) == 6 and read(k=None, fn=fn) == 6
        assert read(dtype=9, fn=fn) == 2 and read(T=-1, fn=fn) == 1 and read(s=-1.0, fn=fn) == 1
        assert read(starts=P(4097), fn=fn) == 3 and read(k=P(4100), fn=fn) == 3 and read(T=0, fn=fn) == 0

    def verify(t=a, d=a, dtype=0, x=a, u=a, B=2, n=4, V=50, tokens=a, acc=a):
        return lib.msa_verify(t, 200, 50, d, 150, 50, dtype, x, u, None, B, n, V, tokens, acc, None)

    def greedy(t=a, dtype=0, x=a, B=2, n=4, V=50, tokens=a, acc=a):
        return lib.msa_verify_greedy(t, 200, 50, dtype, x, None, B, n, V, tokens, acc, None)

    for fn in (verify, greedy):
        assert fn(B=0) == 0
        assert fn(t=None) == 6 and fn(x=None) == 6 and fn(tokens=None) == 6 and fn(acc=None) == 6
        assert fn(dtype=3) == 2
        assert fn(n=0) == 1 and fn(n=33) == 1 and fn(V=0) == 1 and fn(V=2 ** 19) == 1 and fn(B=-1) == 1
        assert fn(t=P(4098)) == 3 and fn(x=P(4097)) == 3 and fn(acc=P(4097)) == 3
    assert verify(u=None) == 6 and verify(d=P(4097)) == 3 and verify(u=P(4097)) == 3


def test_prefix_attention_refusals():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kv = torch.zeros((6, 4, 128), dtype=torch.uint8), torch.zeros((4, 2, 128, 256), dtype=torch.uint8)
    a = {"q": q, "kv": kv, "table": i32(2, 3), "cu_q": i32(3), "cu_k": i32(3), "prefix": 1, "max_q": 6, "max_k": 300}

    def run(**kw):
        c = dict(a, **{k: v for k, v in kw.items() if k in a})
        return _err(msa.msa_prefix_attention, c["q"], c["kv"], 1.0, 1.0, 1.0, 0.1, c["table"], c["cu_q"], c["cu_k"], c["prefix"], c["max_q"], c["max_k"],
                    **{k: v for k, v in kw.items() if k not in a})

    assert "CUDA" in run()
    assert "q has dtype" in run(q=q.to(torch.bfloat16)) and "q must be [any, any, 128]" in run(q=q[0])
    assert "q must be contiguous" in run(q=torch.zeros((6, 8, 128), dtype=torch.uint8)[:, ::2])
    assert "block_table must be" in run(table=i32(3, 3)) and "cu_seqlens_k must be" in run(cu_k=i32(2))
    assert "out must be" in run(out=torch.zeros((6, 2, 128), dtype=torch.bfloat16)) and "lse must be" in run(lse=torch.zeros((6, 3)))
    assert "workspace too small" in run(workspace=torch.zeros(100, dtype=torch.uint8))
    assert "unsupported" in run(q=torch.zeros((6, 3, 128), dtype=torch.uint8))
    assert "unsupported" in run(q=torch.zeros((1, 258, 128), dtype=torch.uint8))
    for bad in (dict(prefix=-1), dict(prefix=3), dict(max_q=-1), dict(max_q=301), dict(max_k=2 ** 30 + 1)):
        assert "out of range" in run(**bad)


def test_prefix_attention_library_refusals():
    lib, P = msa.load(), ctypes.c_void_p
    a = P(4096)

    def run(q=a, kv=a, pages=4, s=1.0, table=a, width=3, cu=a, B=2, T=6, Hq=4, Hkv=2, prefix=1, ws=a, size=1 << 40, out=a, lse=None, status=None):
        return lib.msa_prefix_attention(q, kv, pages, s, 1.0, 1.0, 0.1, table, width, cu, a, B, T, Hq, Hkv, prefix, 6, 300, ws, size, out, lse, status, None)

    assert run(B=0) == 0 and run(T=0) == 0
    assert run(q=None) == 6 and run(kv=None) == 6 and run(table=None) == 6 and run(cu=None) == 6 and run(out=None) == 6
    assert run(width=2) == 1 and run(pages=-1) == 1 and run(pages=2 ** 23) == 1 and run(B=-1) == 1 and run(prefix=-1) == 1
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert run(s=s) == 1
    assert run(s=1e32) == 1 and run(s=1e30, B=0) == 0  # the largest score: 1e32 * 0.1 * log2 e * 128 * 448^2 > 3.4e38
    assert run(Hq=3) == 2 and run(Hq=0) == 1 and run(Hq=258) == 2
    assert run(ws=None) == 4 and run(size=1000) == 4 and run(ws=P(4096 + 128)) == 3
    assert run(q=P(4104)) == 3 and run(out=P(4100)) == 3 and run(lse=P(4098)) == 3 and run(status=P(4097)) == 3
    n = ctypes.c_size_t()
    size = lambda *v: lib.msa_prefix_attention_workspace_bytes(*v, ctypes.byref(n))  # noqa: E731
    assert size(2, 6, 4, 2, 1, 6, 300) == 0 and n.value > 0
    assert size(2, 6, 4, 2, 1, 6, 100) == 1 and size(2, -6, 4, 2, 1, 6, 300) == 1 and size(2, 6, 5, 2, 1, 6, 300) == 2
    assert lib.msa_prefix_attention_workspace_bytes(2, 6, 4, 2, 1, 6, 300, None) == 6


def test_verify_refuses_outputs_over_inputs():
    t, u = torch.zeros((2, 4, 50)), torch.zeros((2, 4))
    room = torch.zeros(20, dtype=torch.int32)
    x, counts = room[:6].view(2, 3), torch.zeros(2, dtype=torch.int32)
    for fn, args in ((msa.msa_verify, (t, x, u)), (msa.msa_verify_greedy, (t, x))):
        for at in (0, 5):
            assert "tokens must not share memory with draft_tokens" in _err(fn, *args, tokens=room[at:at + 8].view(2, 4))
        assert "accepted must not share memory with draft_tokens" in _err(fn, *args, accepted=room[5:7])
        assert "tokens must not share memory with accepted" in _err(fn, *args, tokens=room[6:14].view(2, 4), accepted=room[13:15])
        assert "accepted must not share memory with num_drafts" in _err(fn, *args, num_drafts=room[8:10], accepted=room[9:11])
        assert "CUDA" in _err(fn, *args, tokens=room[6:14].view(2, 4), accepted=counts, num_drafts=counts)
        one = (t[:1], room[:3].view(1, 3), u[:1])[:len(args)]
        assert "CUDA" in _err(fn, *one, tokens=room[:4].view(1, 4))
    assert "tokens must not share memory with uniforms" in _err(msa.msa_verify, t, x, u, tokens=u.view(torch.int32))


def test_prefix_attention_takes_every_length_that_it_documents():
    n = ctypes.c_size_t()
    size = lambda *v: msa.load().msa_prefix_attention_workspace_bytes(*v, ctypes.byref(n))  # noqa: E731
    for B, T, Hq, Hkv, prefix, max_k in ((32, 32, 16, 2, 0, 2 ** 30), (127, 127, 16, 2, 0, 2 ** 30), (1, 2 ** 20, 16, 1, 0, 2 ** 20), (4, 2 ** 15, 128, 1, 8000, 2 ** 20)):
        assert size(B, T, Hq, Hkv, prefix, min(T, max_k), max_k) == 0
        rows = Hkv * (2 if prefix else 1) * T * (Hq // Hkv)
        assert rows * 516 < n.value < (rows + 256 * 200) * 516 + 32 * 2 * (T + B) + 4 * B + 2000
    # either side of n (4 ceil(max_seqlen_k / 128) + 10) < 2^32
    for B, T, Hq, Hkv, prefix in ((128, 128, 16, 2, 0), (5000, 7000, 12, 4, 3), (1, 2 ** 20, 31, 31, 0), (3, 2 ** 18, 128, 1, 1)):
        t = 2 * (128 * Hkv // Hq)
        tiles = min(T, -(-T // t) + B) + (-(-T // t) if prefix else 0)
        pages = min(2 ** 23, ((2 ** 32 - 1) // tiles - 10) // 4)
        assert size(B, T, Hq, Hkv, prefix, 1, 128 * pages) == 0
        assert size(B, T, Hq, Hkv, prefix, 1, 128 * pages + 1) == 1


def test_prefix_attention_sizes_whose_products_wrap():
    n = ctypes.c_size_t()
    for prefix in (2 ** 55, 2 ** 57, 2 ** 57 + 1, 2 ** 62):  # times 128: 2^62, 0, 128 and 0 in 64 bits
        assert msa.load().msa_prefix_attention_workspace_bytes(2, 6, 4, 2, prefix, 6, 300, ctypes.byref(n)) == 1
    a = ctypes.c_void_p(4096)
    for pages in (2 ** 56, 2 ** 57, 2 ** 63 - 1):
        assert msa.load().msa_prefix_attention(a, a, pages, 1.0, 1.0, 1.0, 0.1, a, 3, a, a, 0, 6, 4, 2, 1, 6, 300, a, 1 << 40, a, None, None, None) == 1


def test_nvfp4_write_refuses_a_scale_whose_block_scales_overflow():
    # s = amax / (6 g): 6 g has to be finite in fp32, or every code would be 0
    a = ctypes.c_void_p(4096)

    def run(fn, ks, vs, T=6):
        return fn(a, 256, 128, a, 256, 128, 1, a, 4, ks, vs, a, 3, a, a, 2, T, 2, None, None)

    for big in (5.7e37, 1e38, 3.4e38):
        assert run(msa.load().msa_kv_write_nvfp4, big, 1.0) == 1 and run(msa.load().msa_kv_write_nvfp4, 1.0, big) == 1
        assert run(msa.load().msa_kv_write, big, big, T=0) == 0  # (nothing is launched)
    assert run(msa.load().msa_kv_write_nvfp4, 5.6e37, 5.6e37, T=0) == 0


def test_read_refuses_rows_that_overlap():
    c = _cache()
    run = lambda k, v: _err(msa.msa_kv_read, c["kv"], 1.0, 1.0, c["table"], c["cu_q"], 6, k=k, v=v)  # noqa: E731
    room = torch.zeros(6 * 2 * 256 + 256)
    rows = lambda at, token, head: room.as_strided((6, 2, 128), (token, head, 1), at)  # noqa: E731
    good = rows(0, 512, 256)
    for bad in (rows(0, 0, 128), rows(0, 512, 0), rows(0, 64, 512), rows(0, 128, 128), rows(0, 256, 192), rows(0, 256, 256)):
        assert "rows of k must not overlap" in run(bad, torch.zeros(6, 2, 128)) and "rows of v must not overlap" in run(torch.zeros(6, 2, 128), bad)
    assert "k and v must not share rows" in run(good, good)
    for k, v in ((good, rows(128, 512, 256)), (rows(0, 256, 128), torch.zeros(6, 2, 128)), (rows(0, 128, 768), rows(1536, 128, 768))):
        assert "CUDA" in run(k, v)
