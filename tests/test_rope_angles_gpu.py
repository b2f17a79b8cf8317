"""The rotation's angles where their errors show: cosines and sines near 0, at
positions near 2^31.

An angle in (-1/2, 1/2] turns is rounded to 2^-32 turns (off by 2^-33, with the
frequency's own 2^-65 a position less than 2^-32) and then to fp32, 2^-26 at half a
turn and 2^-27 at a quarter.  Near these a sine or cosine is 2 pi times the
distance, and its own rounding is one of itself."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


@pytest.mark.parametrize("freq", [1.0, 0.7, 5.5, 2 * math.pi / 7, 1e-3])
def test_components_near_zero(freq):
    pos = np.arange(2 ** 31 - 2 * 10 ** 6, 2 ** 31 - 1, dtype=np.int64)
    turn = (pos.astype(np.uint64) * np.uint64(msa.msa_rope_turns([freq])[0])) / 2.0 ** 64
    near = np.abs((turn * 4 + 0.5) % 1 - 0.5) < 4e-5  # quarters, halves and whole turns
    pos = pos[near][:512]
    assert len(pos) > 100
    q = torch.zeros((len(pos), 1, 128), device="cuda")
    q[..., 0] = 1
    kv = torch.zeros((8, 1, 128, 256), dtype=torch.uint8, device="cuda")
    table, cu = torch.arange(8, dtype=torch.int32, device="cuda")[None], torch.tensor([0, len(pos)], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        got = msa.msa_rope_write(msa.MsaRope([freq], interleaved=interleaved), q, q, q, kv, None, 1.0, 1.0, table, cu, cu,
                                 positions=torch.from_numpy(pos.astype(np.int32)).cuda())[:, 0, :2].double().cpu().numpy()
        for p, (c, s) in zip(pos.tolist(), got):
            x = Fraction(p) * Fraction(freq) / (2 * PI) % 1
            quarter = int(x * 4 + Fraction(1, 2))
            angle = float((x - Fraction(quarter, 4)) * 2 * PI)  # from the nearest quarter
            a, b = math.cos(angle), math.sin(angle)
            want = [(a, b), (-b, a), (-a, -b), (b, -a)][quarter % 4]
            for g, w in zip((c, s), want):
                assert abs(g - w) <= 2.0 ** -8 * abs(w) + 2 * math.pi * (2.0 ** -26 + 2.0 ** -32), (p, g, w)
