"""The NVFP4 codes and block scales of K as msa_rope_write_nvfp4 writes them, each
one by itself, against formulas in 64 bits.

A value before its quantisation is off by less than 2^-20 (|a| + |b|) (as derived
in test_rope_write_gpu.py), and the fp32 quotients that are rounded to codes by
2^-22 of themselves.  Rounding is monotone, so a block's scale lies between the
scales of the smallest and the largest amax within that, and a code, by the scale
that was written, between those of the smallest and the largest value."""
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_rope_write_gpu import CASES, EPS, KS, QS, VS, Batch, _turned, _value8

pytestmark = pytest.mark.gpu

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _nearest4(x):
    """E2M1 values nearest to x (fp64), even codes on ties, saturating."""
    grid = E2M1.to(x.device)
    mag = x.abs()
    mid = (grid[1:] + grid[:-1]) / 2
    code = (mag[..., None] > mid).sum(-1)
    tie = (mag[..., None] == mid) & (torch.arange(7, device=x.device) % 2 == 1)  # between an odd code and the next: up
    return torch.copysign(grid[code + tie.any(-1)], x)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES)
def test_every_written_code_and_scale(case, dtype):
    q_lens, seqs, hq, hkv, pairs, interleaved, axes, norm = case
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    freq = (1e4 ** -(torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).tolist()
    axis = [j % axes for j in range(pairs)]
    w = 1 + 0.3 * torch.randn((2, 128), generator=g, device="cuda")
    s = Batch(q_lens, seqs, hq, hkv, dtype, True, seed=3, pad=2)
    positions = torch.randint(-50, 1100000, (axes, s.T), generator=g, device="cuda", dtype=torch.int32)
    rope = msa.MsaRope(freq, interleaved=interleaved, axes=axis if axes > 1 else None, q_norm=w[0] if norm else None, k_norm=w[1] if norm else None, eps=EPS)
    before = s.kv.clone()
    msa.msa_rope_write_nvfp4(rope, s.q if hq else None, s.k, s.v, s.kv, QS, KS, VS, s.table, s.cu_q, s.cu_k, positions=positions)
    k, size = (t[:s.n] for t in _turned(s.k, w[1] if norm else None, positions, axis, freq, interleaved))
    page, row = s.where()
    code_at = row[:, None] * 64 + torch.arange(64, device="cuda")
    scale_at = 8192 + row[:, None] * 8 + torch.arange(8, device="cuda")
    slot = s.kv[page, :, 0]  # [n, hkv, 9216]
    bytes4 = slot.gather(2, code_at[:, None].expand(-1, hkv, -1))
    scales = slot.gather(2, scale_at[:, None].expand(-1, hkv, -1))
    err = 2.0 ** -20 * size
    blocks = lambda t: t.reshape(s.n, hkv, 8, 16)  # noqa: E731
    g6 = 6.0 * float(torch.tensor(KS, dtype=torch.float32))
    amax = lambda t: (blocks(t.clamp(min=0)).amax(-1) / g6)  # noqa: E731
    lo, hi = amax(k.abs() - err) * (1 - 2.0 ** -22), amax(k.abs() + err) * (1 + 2.0 ** -22)
    code8 = lambda t: _value8(t.clamp(max=448).float().to(torch.float8_e4m3fn).view(torch.uint8))  # noqa: E731
    got8 = _value8(scales)
    assert ((got8 >= code8(lo)) & (got8 <= code8(hi))).all()
    den = (got8 * (g6 / 6)).clamp(min=1e-300)[..., None]
    lo, hi = blocks(k - err) / den, blocks(k + err) / den
    lo, hi = _nearest4(lo - 2.0 ** -22 * lo.abs()), _nearest4(hi + 2.0 ** -22 * hi.abs())
    nibbles = torch.stack([bytes4 & 15, bytes4 >> 4], -1).reshape(s.n, hkv, 128).long()
    got4 = blocks(torch.where(nibbles >= 8, -1.0, 1.0) * E2M1.cuda()[nibbles & 7])
    zero = (got8 == 0)[..., None]
    assert (torch.where(zero, got4 == 0, (got4 >= lo) & (got4 <= hi))).all()
    # V's slot is that of msa_kv_write, and no other byte has changed
    other = before.clone()
    msa.msa_kv_write_nvfp4(s.k, s.v, other, KS, VS, s.table, s.cu_q, s.cu_k)
    assert torch.equal(s.kv[:, :, 1], other[:, :, 1])
    for h in range(hkv):
        for at in (code_at, scale_at):
            before[page[:, None], h, 0, at] = s.kv[page[:, None], h, 0, at]
    assert torch.equal(s.kv[:, :, 0], before[:, :, 0])


def test_nearest_codes():
    x = torch.tensor([0.24, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 9.0, -0.75], dtype=torch.float64, device="cuda")
    assert _nearest4(x).tolist() == [0, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, -1]
