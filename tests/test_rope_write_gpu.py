"""Rotation with the cache write against formulas in 64 bits.

Tolerances of the values before their last rounding, from the roundings: the
angle is off by less than 2^-31 of a turn (in 32 bits of a turn, then as an
fp32 number: 2^-25 of a half turn), so cosine and sine by less than 2^-22 with
their own rounding; a pair's sum has three roundings of 2^-24 of |a| + |b|, the
norm adds at most eight of x (the sum of 128 squares in pairs, a root and a
division).  Together less than 2^-20 (|a| + |b|) w.  A code's value is then off
by half a step more: 2^-4 of it or 2^-10 (E4M3 below its normal values); bf16
by 2^-8."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

QS, KS, VS = 0.0131, 0.0127, 0.0149
EPS = 1e-6


def _value8(c):
    return c.view(torch.float8_e4m3fn).double()


def _turned(x, w, positions, axes, freq, interleaved):
    """(rows in 64 bits, the bound's |a| + |b|)."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    n = len(freq)
    y, size = x.clone(), x.abs()
    if n:
        pos = positions.double().reshape(-1, x.shape[0])
        angle = pos[torch.tensor(axes, device="cuda")].T * torch.tensor(freq, dtype=torch.float64, device="cuda")
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * c - b * s, a * s + b * c
        size[..., i] = size[..., j] = a.abs() + b.abs()
    return y, size


def _near_e4m3(code, want, size, scale):
    """Codes of want / scale, `size` the bound of what want was computed from."""
    got = _value8(code)
    w = want / scale
    err = 2.0 ** -20 * size / scale
    lo, hi = (w - err).clamp(-448, 448), (w + err).clamp(-448, 448)
    half = torch.maximum(2.0 ** -4 * torch.maximum(lo.abs(), hi.abs()), torch.tensor(2.0 ** -10, device="cuda"))
    bad = (got < lo - half) | (got > hi + half)
    assert not bad.any(), (bad.sum().item(), got[bad][:4], w[bad][:4])


class Batch:
    def __init__(self, q_lens, seqs, hq, hkv, dtype, fp4, seed=0, pad=0, fused=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.T = sum(q_lens) + pad
        x = torch.randn((self.T, hq + 2 * hkv, 128), generator=g, device="cuda").to(dtype)
        if fused:
            self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        else:
            self.q, self.k, self.v = (p.clone(memory_format=torch.contiguous_format) for p in (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]))
        pages = [-(-s // 128) for s in seqs]
        perm = np.random.RandomState(seed).permutation(sum(pages) + 2).astype(np.int32)
        table = np.full((len(seqs), max(pages + [1])), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.kv = torch.full((sum(pages) + 2, hkv) + ((2, 9216) if fp4 else (128, 256)), 0x5A, dtype=torch.uint8, device="cuda")
        cu = lambda v: torch.from_numpy(np.concatenate([[0], np.cumsum(v)]).astype(np.int32)).cuda()  # noqa: E731
        self.cu_q, self.cu_k = cu(q_lens), cu(seqs)
        self.n = sum(q_lens)
        self.place = torch.cat([torch.arange(m - n, m) for n, m in zip(q_lens, seqs)]).cuda()
        self.b = torch.repeat_interleave(torch.arange(len(seqs)), torch.tensor(q_lens)).cuda()

    def where(self):
        return self.table.long()[self.b, self.place // 128], self.place % 128


CASES = [
    # q_lens, seqs, hq, hkv, pairs, interleaved, axes, norm
    ([1], [1], 1, 1, 64, False, 1, False),
    ([1], [129], 16, 1, 64, True, 1, True),
    ([8] * 5, [8, 100, 128, 131, 4000], 16, 2, 32, False, 1, True),
    ([3, 0, 7, 1], [300, 20, 7, 65], 6, 2, 48, False, 3, True),
    ([5, 130], [5, 257], 5, 1, 10, False, 1, True),
    ([33], [40], 12, 4, 40, False, 1, False),
    ([33], [40], 12, 4, 1, False, 2, True),
    ([17, 200], [30, 200], 6, 3, 37, True, 8, False),
    ([64], [64], 2, 2, 0, False, 1, True),
    ([700, 1], [900, 1000], 40, 8, 64, False, 1, True),
    ([2000], [2000], 0, 3, 64, False, 1, False),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES)
def test_matches_formulas(case, dtype):
    q_lens, seqs, hq, hkv, pairs, interleaved, axes, norm = case
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    freq = (1e4 ** -(torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).tolist()
    axis = [j % axes for j in range(pairs)]
    w = 1 + 0.3 * torch.randn((2, 128), generator=g, device="cuda")
    for fp4, bf16, pad in ((False, False, 0), (True, True, 3), (False, True, 0), (True, False, 0)):
        s = Batch(q_lens, seqs, hq, hkv, dtype, fp4, pad=pad, fused=not bf16)
        rope = msa.MsaRope(freq, interleaved=interleaved, axes=axis if axes > 1 else None, q_norm=w[0] if norm else None, k_norm=w[1] if norm else None, eps=EPS)
        positions = torch.randint(-50, 1100000, (axes, s.T), generator=g, device="cuda", dtype=torch.int32) if axes > 1 or pad else None
        at = torch.nn.functional.pad(s.place, (0, pad)) if positions is None else positions
        before = s.kv.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full((s.T, hq, 128), 7.0, device="cuda").to(torch.bfloat16 if bf16 else torch.float8_e4m3fn) if hq else None
        fn = msa.msa_rope_write_nvfp4 if fp4 else msa.msa_rope_write
        keep = None if q_out is None else q_out.clone()
        got = fn(rope, s.q if hq else None, s.k, s.v, s.kv, None if bf16 else QS, KS, VS, s.table, s.cu_q, s.cu_k,
                 positions=positions if axes > 1 or positions is None else positions[0], q_out=q_out, status=status)
        assert status.item() == 0 and got is q_out
        if hq:
            want, size = _turned(s.q, w[0] if norm else None, at, axis, freq, interleaved)
            if bf16:
                err = (got.double() - want).abs()[:s.n]
                assert (err <= 2.0 ** -8 * want.abs()[:s.n] + 2.0 ** -19 * size[:s.n]).all()
            else:
                _near_e4m3(got[:s.n], want[:s.n], size[:s.n], QS)
            assert torch.equal(got[s.n:].view(torch.uint8), keep[s.n:].view(torch.uint8))
        k, size = _turned(s.k, w[1] if norm else None, at, axis, freq, interleaved)
        page, row = s.where()
        if fp4:
            # V's bytes are those of msa_kv_write; K's those of it for a K that
            # is turned already, wherever no code lies at a border: the values
            # read back are compared, with the block's step (s 2 at most between
            # codes, s <= amax / 6 (1 + 2^-3)) and the rounding to E4M3
            other = before.clone()
            msa.msa_kv_write_nvfp4(k.float()[:s.n], s.v.float()[:s.n], other, KS, VS, s.table, s.cu_q, s.cu_k)
            assert torch.equal(s.kv[:, :, 1], other[:, :, 1])
            a, b = msa.msa_nvfp4_to_e4m3(s.kv).double()[page, :, row, :128] * KS, k[:s.n]
            amax = b.abs().reshape(*b.shape[:-1], 8, 16).amax(-1).repeat_interleave(16, -1)
            assert ((a - b).abs() <= amax * (1 / 6 * 1.125 + 2.0 ** -4) + 2.0 ** -9 * KS).all()
            same = (s.kv[:, :, 0] == other[:, :, 0]).double().mean().item()
            assert same > 0.99
        else:
            _near_e4m3(s.kv[page, :, row, :128], k[:s.n], size[:s.n], KS)
            other = before.clone()
            msa.msa_kv_write(s.k[:s.n], s.v[:s.n], other, KS, VS, s.table, s.cu_q, s.cu_k)
            assert torch.equal(s.kv[..., 128:], other[..., 128:])
            other[page, :, row] = s.kv[page, :, row]
            assert torch.equal(other, s.kv)  # nothing but the new rows changed


def test_far_positions_turn_exactly():
    """At positions near 2^31 the angle still is right to 2^-31 turns."""
    s = Batch([64], [64], 1, 1, torch.float32, False)
    freq = [1.0, 0.7, 3.0, 1e-3, 2 * np.pi / 7, 5.5]
    pos = torch.randint(2 ** 31 - 10 ** 6, 2 ** 31 - 1, (64,), dtype=torch.int32, device="cuda")
    s.q.zero_()
    s.q[..., 0:12:2] = 1.0
    q = msa.msa_rope_write(msa.MsaRope(freq, interleaved=True), s.q, s.k, s.v, s.kv, None, KS, VS, s.table, s.cu_q, s.cu_k, positions=pos)
    # angles by whole numbers: pos * round(2^80 f / 2 pi), exact enough by 2^-48 turns
    from fractions import Fraction
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    for j, f in enumerate(freq):
        turn = [float((Fraction(p) * Fraction(f) / (2 * pi)) % 1) for p in pos.tolist()]
        want = torch.tensor([[np.cos(2 * np.pi * x), np.sin(2 * np.pi * x)] for x in turn], device="cuda")
        got = q[:, 0, 2 * j:2 * j + 2].double()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20).all()


@pytest.mark.parametrize("fp4", [False, True])
def test_special_values(fp4):
    """NaN and infinities stay in their pair; what is not rotated is as msa_kv_write writes it."""
    s = Batch([20], [150], 2, 2, torch.bfloat16, fp4)
    s.k[3, 0, 5] = float("nan")
    s.k[4, 1, 100] = float("inf")
    s.q[5, 1, 127] = float("nan")
    freq = [1.0 / (j + 1) for j in range(48)]
    q = msa.msa_rope_write_nvfp4 if fp4 else msa.msa_rope_write
    out = q(msa.MsaRope(freq), s.q, s.k, s.v, s.kv, QS, KS, VS, s.table, s.cu_q, s.cu_k)
    nan = torch.isnan(out.float())
    assert nan.sum() == 1 and nan[5, 1, 127]
    page, row = s.where()
    other = torch.full_like(s.kv, 0x5A)
    (msa.msa_kv_write_nvfp4 if fp4 else msa.msa_kv_write)(s.k, s.v, other, KS, VS, s.table, s.cu_q, s.cu_k)
    if not fp4:
        assert torch.equal(s.kv[page, :, row, 96:128], other[page, :, row, 96:128])
        got = torch.isnan(s.kv.view(torch.float8_e4m3fn).float()[page, :, row, :128])
        assert got.sum() == 2 and got[3, 0, 5] and got[3, 0, 53]


def test_bad_tokens_are_left_out():
    """A page that is none, lengths that do not fit: their tokens, Q with them, are not written."""
    s = Batch([4, 4, 4], [10, 200, 4], 2, 1, torch.bfloat16, False)
    s.table[1, 1] = 10 ** 6
    s.cu_k[3] = s.cu_k[2] + 2  # fewer than the request's new tokens
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = s.kv.clone()
    out = torch.full((12, 2, 128), 3, dtype=torch.uint8, device="cuda")
    msa.msa_rope_write(msa.MsaRope([1.0, 0.1]), s.q, s.k, s.v, s.kv, QS, KS, VS, s.table, s.cu_q, s.cu_k, q_out=out, status=status)
    assert status.item() == msa.STATUS_BAD_BLOCK | msa.STATUS_BAD_SEQLENS
    assert (out[:4] != 3).any() and (out[4:] == 3).all()
    assert int((s.kv != before).any(-1).sum()) == 4


def test_graph_and_other_stream():
    s = Batch([3] * 600, [130] * 600, 4, 1, torch.bfloat16, False)  # more requests than are staged
    rope = msa.MsaRope([1.0 / (j + 1) for j in range(64)], q_norm=torch.ones(128, device="cuda"))
    call = lambda **kw: msa.msa_rope_write(rope, s.q, s.k, s.v, s.kv, QS, KS, VS, s.table, s.cu_q, s.cu_k, **kw)  # noqa: E731
    want, pool = call(), s.kv.clone()
    side = torch.cuda.Stream()
    s.kv.fill_(0x5A)
    torch.cuda.synchronize()
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s.kv, pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    s.kv.fill_(0x5A)
    graph.replay()
    assert torch.equal(out.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s.kv, pool)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rounds_of_ctas(dtype, fp4):
    """Numbers of tokens around whole rounds of the GPU's places, whose last round is split another way: the same bytes as in small calls."""
    tokens = torch.cuda.get_device_properties(0).multi_processor_count * 4 * (4 if fp4 else 5) * (2 if dtype == torch.float32 else 4)
    heads, most = (3, 2), 2 * tokens + tokens // 3 + 1
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((most, heads[0] + 2 * heads[1], 128), generator=g, device="cuda").to(dtype)
    q, k, v = x[:, :3], x[:, 3:5], x[:, 5:]
    pages = -(-most // 128)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    rope = msa.MsaRope([0.8 ** j for j in range(64)], q_norm=torch.rand(128, generator=g, device="cuda"), k_norm=torch.rand(128, generator=g, device="cuda"))
    write = msa.msa_rope_write_nvfp4 if fp4 else msa.msa_rope_write
    new = lambda: torch.zeros((pages, 2, 2, 9216) if fp4 else (pages, 2, 128, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, parts = new(), []
    for a in range(0, most, 1000):
        b = min(a + 1000, most)
        parts.append(write(rope, q[a:b], k[a:b], v[a:b], pool, QS, KS, VS, table, i32([0, b - a]), i32([0, b])))
    parts = torch.cat(parts).view(torch.uint8)
    for T in (tokens // 7 + 1, tokens // 2 + 2, tokens - 1, tokens, tokens + 1, tokens + tokens // 2, 2 * tokens - 3, most):
        got, status = new(), i32([0])
        out = write(rope, q[:T], k[:T], v[:T], got, QS, KS, VS, table, i32([0, T]), i32([0, T]), status=status)
        assert status.item() == 0 and torch.equal(out.view(torch.uint8), parts[:T])
        want = pool.clone()
        if T < most:  # rows behind the last stay as they were
            page, off = T // 128, T % 128
            keep = table[0, :page].long()
            clean = new()
            clean[keep] = pool[keep]
            if off:
                last = int(table[0, page])
                if fp4:
                    clean[last, :, :, :off * 64] = pool[last, :, :, :off * 64]
                    clean[last, :, :, 8192:8192 + off * 8] = pool[last, :, :, 8192:8192 + off * 8]
                else:
                    clean[last, :, :off] = pool[last, :, :off]
            want = clean
        assert torch.equal(got, want)


@pytest.mark.parametrize("scale", [0.01, 0.02, 0.05, 0.1, 1 / 3, 0.7, 1.9999999, 3.0, 1e-8, 1.1e-25, 1e-27, 1e20, 0.25, 0.0131])
def test_codes_are_of_the_rounded_quotient(scale):
    """Codes of values near the middle of two codes: V's, and K's of msa_kv_write, are E4M3 of the fp32 quotient."""
    s32 = float(np.float32(scale))
    codes = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()
    mid = ((codes[1:] + codes[:-1]) / 2).double() * s32
    near = mid.float().view(torch.int32)[:, None] + torch.arange(-40, 41, device="cuda", dtype=torch.int32)
    every = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.uint16)
    for x in (near.flatten().view(torch.float32), every.view(torch.bfloat16), every.view(torch.float16)):
        x = torch.cat([x, -x])
        T = -(-x.numel() // 128)
        v = torch.nn.functional.pad(x, (0, T * 128 - x.numel())).view(T, 1, 128)
        want = (v.float() / torch.full_like(v, s32, dtype=torch.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pages = T // 128 + 1
        table, cu = torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.tensor([0, T], dtype=torch.int32, device="cuda")
        nan = torch.isnan(v.float())
        for write in (lambda kv: msa.msa_rope_write(msa.MsaRope([]), None, torch.zeros_like(v), v, kv, 1.0, 1.0, s32, table, cu, cu),
                      lambda kv: msa.msa_kv_write(v, v, kv, s32, s32, table, cu, cu)):
            kv = torch.zeros((pages, 1, 128, 256), dtype=torch.uint8, device="cuda")
            write(kv)
            got = kv.view(-1, 256)[:T, 128:].reshape(T, 1, 128)
            assert torch.equal(got[~nan], want[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()
