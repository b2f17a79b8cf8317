"""Cache writes and reads against plain numpy.

Writes are compared code for code: a code is the nearest E4M3 (E2M1) value to
a quotient taken in fp32, which numpy takes the same way, so the codes are
equal, and against 64 bits a code is off by at most half a step.  Reads are
compared with the product of code and scale in fp32, rounded to the type:
equal too.  Whole pools and whole outputs are compared, so that a row written
where none belongs is seen."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
import oracle

pytestmark = pytest.mark.gpu

TYPES = (torch.float32, torch.bfloat16, torch.float16)
SLOT, CODES = msa.NVFP4_SLOT_BYTES, 128 * 64


def _e4m3_values():
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e > 0, 2.0 ** (e - 7.0) * (1 + m / 8.0), m * 2.0 ** -9)
    v = np.where(c & 0x80, -v, v)
    v[(c & 0x7F) == 0x7F] = np.nan
    return v


E4M3 = _e4m3_values()
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _nearest(x, grid):
    """Index of the nearest value of an ascending grid to |x| (float64 of an
    fp32 number), ties to the even index, the ends saturating."""
    a = np.abs(x.astype(np.float64))
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def _to_e4m3(x):
    code = _nearest(np.nan_to_num(x, nan=0.0, posinf=1e30, neginf=-1e30), E4M3[:0x7F]).astype(np.uint8)
    code |= np.signbit(x).astype(np.uint8) << 7
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def _to_nvfp4(x, g):
    """fp32 [..., 128] -> code bytes [..., 64], block scales [..., 8]."""
    xb = x.reshape(*x.shape[:-1], 8, 16)
    with np.errstate(all="ignore"):
        amax = np.nanmax(np.where(np.isnan(xb), 0, np.abs(xb)), axis=-1)
        scale = _to_e4m3(amax / (np.float32(6) * np.float32(g)))
        den = (E4M3[scale].astype(np.float32) * np.float32(g))[..., None]
        y = np.where(den > 0, xb / den, np.float32(0)).astype(np.float32)
        y = np.nan_to_num(y, nan=0.0, posinf=1e30, neginf=-1e30)
    code = _nearest(y, E2M1) | (np.signbit(y) << 3)
    # a NaN or a block without a scale is written as +0
    code = np.where(np.isnan(xb) | (den == 0), 0, code).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def _batch(q_lens, seqs, seed, spare=2):
    r = np.random.RandomState(seed)
    need = [-(-s // 128) for s in seqs]
    pages = sum(need) + spare
    perm = r.permutation(pages).astype(np.int32)
    table = np.full((len(seqs), max(need + [1])), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = lambda v: np.concatenate([[0], np.cumsum(v)]).astype(np.int32)  # noqa: E731
    return table, pages, cu(q_lens), cu(seqs)


def _rows(table, first, lens):
    """(page, row in it) of `lens[b]` positions from first[b] on, by request."""
    page, row = [], []
    for b, (f, n) in enumerate(zip(first, lens)):
        pos = np.arange(f, f + n)
        page.append(table[b, pos // 128])
        row.append(pos % 128)
    return np.concatenate(page).astype(np.int64), np.concatenate(row)


def _values(shape, r):
    x = r.standard_normal(shape).astype(np.float32) * np.exp2(r.uniform(-12, 9, shape[:-1] + (1,))).astype(np.float32)
    f = x.reshape(-1)
    for i, v in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-30, -1e-30, 3e38)):
        if f.size > 137 * i + 5:
            f[137 * i + 5] = v
    return x


BATCHES = [
    # q_lens, sequence lengths, heads
    ([1], [1], 1),
    ([1], [128], 2),
    ([3, 0, 1, 129], [3, 77, 129, 400], 3),
    ([8] * 64, [100 + 37 * b for b in range(64)], 2),
    ([1] * 1100, [1 + b % 260 for b in range(1100)], 1),
    ([1000, 1, 257], [1000, 5000, 300], 8),
    ([5, 0, 0], [130, 0, 9], 127),
]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("fp4", [False, True], ids=["e4m3", "nvfp4"])
@pytest.mark.parametrize("case", range(len(BATCHES)))
def test_write_then_read(case, fp4, dtype):
    q_lens, seqs, H = BATCHES[case]
    r = np.random.RandomState(case)
    table, pages, cu_q, cu_k = _batch(q_lens, seqs, case)
    T = int(cu_q[-1])
    ks, vs = 0.0123, 0.71
    # K and V as parts of a wider row, and two rows of padding behind the batch
    wide = torch.from_numpy(_values((T + 2, 3, H, 128), r)).to("cuda").to(dtype)
    k, v = wide[:, 2], wide[:, 0]
    shape = (pages, H, 2, SLOT) if fp4 else (pages, H, 128, 256)
    before = r.randint(0, 256, shape, dtype=np.uint8)
    if fp4:  # finite block scales, as the format has them
        sc = before[..., CODES:]
        sc[(sc & 0x7F) == 0x7F] ^= 1
    pool = torch.from_numpy(before).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    write = msa.msa_kv_write_nvfp4 if fp4 else msa.msa_kv_write
    write(k, v, pool, ks, vs, dev(table), dev(cu_q), dev(cu_k), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    first = [s - n for s, n in zip(seqs, q_lens)]
    page, row = _rows(table, first, q_lens)
    want = before.copy()
    with np.errstate(all="ignore"):
        for half, x, s in ((0, k, ks), (1, v, vs)):
            x = x[:T].float().cpu().numpy()
            if fp4:
                codes, scale = _to_nvfp4(x, s)
                want[:, :, half, :CODES].reshape(pages, H, 128, 64)[page, :, row] = codes
                want[:, :, half, CODES:].reshape(pages, H, 128, 8)[page, :, row] = scale
            else:
                code = _to_e4m3(x / np.float32(s))
                want[page, :, row, half * 128:half * 128 + 128] = code
                # against 64 bits: half a step, 2^-4 of the value, and the
                # fp32 quotient's own 2^-24 (2^-10: half a subnormal step)
                y = x.astype(np.float64) / np.float64(np.float32(s))
                ok = np.isfinite(y) & (np.abs(y) <= 448)
                err = np.abs(E4M3[code] - y)[ok]
                assert (err <= np.abs(y[ok]) * (2.0 ** -4 + 2.0 ** -23) + 2.0 ** -10).all()
    assert np.array_equal(pool.cpu().numpy(), want)

    # and back: everything of every request from position 0 on, one row more
    # than that in the outputs, which keeps what it held
    read = msa.msa_kv_read_nvfp4 if fp4 else msa.msa_kv_read
    n = int(cu_k[-1])
    out = torch.full((n + 1, H, 2, 128), 7.0, dtype=dtype, device="cuda")
    read(pool, ks, vs, dev(table), dev(cu_k), n + 1, k=out[:, :, 1], v=out[:, :, 0], status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    page, row = _rows(table, [0] * len(seqs), seqs)
    e4 = oracle.nvfp4_to_e4m3(torch.from_numpy(want)) if fp4 else want
    for half, x, s in ((0, out[:, :, 1], ks), (1, out[:, :, 0], vs)):
        f = E4M3[e4[page, :, row, half * 128:half * 128 + 128]].astype(np.float32) * np.float32(s)
        ref = torch.from_numpy(f).to(dtype)
        got = x[:n].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))
        assert (x[n:] == 7.0).all()


@pytest.mark.parametrize("fp4", [False, True], ids=["e4m3", "nvfp4"])
def test_read_from_odd_starts(fp4):
    seqs, starts, lens = [700, 1, 300, 129], [13, 0, 128, 127], [600, 1, 0, 2]
    table, pages, _, _ = _batch(lens, seqs, 5)
    r = np.random.RandomState(5)
    raw = r.randint(0, 256, (pages, 2, 2, SLOT) if fp4 else (pages, 2, 128, 256), dtype=np.uint8)
    if fp4:
        sc = raw[..., CODES:]
        sc[(sc & 0x7F) == 0x7F] ^= 1
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    read = msa.msa_kv_read_nvfp4 if fp4 else msa.msa_kv_read
    k, v = read(torch.from_numpy(raw).cuda(), 2.0, 0.5, torch.from_numpy(table).cuda(), cu, sum(lens),
                starts=torch.tensor(starts, dtype=torch.int32).cuda(), dtype=torch.float32)
    page, row = _rows(table, starts, lens)
    e4 = oracle.nvfp4_to_e4m3(torch.from_numpy(raw)) if fp4 else raw
    for half, x, s in ((0, k, 2.0), (1, v, 0.5)):
        want = E4M3[e4[page, :, row, half * 128:half * 128 + 128]].astype(np.float32) * np.float32(s)
        assert np.array_equal(x.cpu().numpy(), want, equal_nan=True)


def test_bad_pages_and_lengths_are_left_out():
    H, pages = 2, 9
    k = torch.ones((12, H, 128), dtype=torch.bfloat16, device="cuda")
    # request 0: a table entry outside the pool, request 1: -1, request 2:
    # more new tokens than its length, request 3: a position past its row of
    # the table, request 4: in order
    cu_q = torch.tensor([0, 2, 4, 6, 8, 12], dtype=torch.int32).cuda()
    cu_k = torch.tensor([0, 2, 4, 5, 400, 404], dtype=torch.int32).cuda()
    table = torch.tensor([[pages, 0], [-1, 0], [1, 1], [2, 3], [4, 5]], dtype=torch.int32).cuda()
    for fp4 in (False, True):
        pool = torch.zeros((pages, H, 2, SLOT) if fp4 else (pages, H, 128, 256), dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        (msa.msa_kv_write_nvfp4 if fp4 else msa.msa_kv_write)(k, k, pool, 1.0, 1.0, table, cu_q, cu_k, status=status)
        assert status.item() == msa.STATUS_BAD_BLOCK | msa.STATUS_BAD_SEQLENS
        touched = pool.flatten(1).any(1).nonzero().flatten().tolist()
        assert touched == [4]
        status.zero_()
        out = torch.full((12, H, 128), 3.0, device="cuda")
        o2 = out.clone()
        starts = torch.tensor([0, 5, -1, 255, 0], dtype=torch.int32).cuda()
        (msa.msa_kv_read_nvfp4 if fp4 else msa.msa_kv_read)(pool, 1.0, 1.0, table, cu_q, 12, starts=starts, k=out, v=o2, status=status)
        assert status.item() == msa.STATUS_BAD_BLOCK | msa.STATUS_BAD_SEQLENS
        # request 2's position -1 is left out and its position 0 read (page 1:
        # zeros), request 3's 255 read and 256 left out, request 4 read
        want = torch.full((12,), 3.0)
        want[5] = want[6] = 0.0
        want[8:12] = 1.0
        assert torch.equal(out.cpu(), want[:, None, None].expand(12, H, 128))
        assert torch.equal(o2, out)


def test_offsets_beyond_32_bits():
    pages, H = 70000, 2  # 4.6 GB
    pool = torch.empty((pages, H, 128, 256), dtype=torch.uint8, device="cuda")
    x = torch.randn((130, H, 128), device="cuda")
    table = torch.tensor([[69999, 3]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 130], dtype=torch.int32).cuda()
    pool[3].zero_()
    msa.msa_kv_write(x, 2 * x, pool, 0.01, 0.02, table, cu, cu)
    k, v = msa.msa_kv_read(pool, 0.01, 0.02, table, cu, 130, dtype=torch.float32)
    assert torch.equal(k * 2, v)
    x = x.clamp(-4.48, 4.48)  # codes saturate at 448: 448 * 0.01; about 0.2 values of |x| > 4.48 are expected among 33280 normal ones
    assert ((k - x).abs() <= x.abs() * 2.0 ** -4 + 0.01 * 2.0 ** -10).all()
    assert not pool[3, :, 2:].any()


def test_other_stream_and_graph():
    q_lens, seqs, H = [8] * 5, [200, 8, 129, 500, 64], 2
    table, pages, cu_q, cu_k = (torch.from_numpy(a).cuda() if isinstance(a, np.ndarray) else a for a in _batch(q_lens, seqs, 1))
    pool = torch.zeros((pages, H, 128, 256), dtype=torch.uint8, device="cuda")
    k = torch.zeros((40, H, 128), dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([s - 8 for s in seqs], dtype=torch.int32).cuda()
    out = torch.empty_like(k), torch.empty_like(k)

    def step(stream=None):
        msa.msa_kv_write(k, k, pool, 0.02, 0.02, table, cu_q, cu_k, stream=stream)
        msa.msa_kv_read(pool, 0.02, 0.02, table, cu_q, 40, starts=starts, k=out[0], v=out[1], stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    k.copy_(torch.randn_like(k))
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    want = [o.clone() for o in out]
    assert want[0].any()
    got = msa.msa_kv_read(pool, 0.02, 0.02, table, cu_q, 40, starts=starts, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    k.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], -want[0]) and torch.equal(out[1], -want[1])
