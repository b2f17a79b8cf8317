"""Scales of the rotation's E4M3 codes of Q and K: those without a finite
reciprocal are refused, all others give the quotient's code or, where it lies
within 2^-21 of the middle of two, its neighbour's."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa


def test_scales_without_a_finite_reciprocal_are_refused():
    lib, a = msa.load(), ctypes.c_void_p(4096)  # never dereferenced: T is 0
    s = msa.MsaRopeStruct()
    s.axes = 1

    def run(fn, ks=1.0, qs=1.0, vs=1.0, bf16=0, Hq=4):
        return fn(ctypes.addressof(s), None, a, 512, 128, a, 256, 128, a, 256, 128, 1, a, bf16, qs, a, 4, ks, vs, a, 3, a, a, 2, 0, Hq, 2, None, None)

    for tiny in (1e-39, 1.4e-45, 2.9e-39):
        assert run(lib.msa_rope_write, ks=tiny) == 1 and run(lib.msa_rope_write, qs=tiny) == 1 and run(lib.msa_rope_write_nvfp4, qs=tiny) == 1
        # where no code comes from a reciprocal
        assert run(lib.msa_rope_write, vs=tiny) == 0 and run(lib.msa_rope_write_nvfp4, ks=tiny) == 0
        assert run(lib.msa_rope_write, qs=tiny, bf16=1) == 0 and run(lib.msa_rope_write, qs=tiny, Hq=0) == 0
    assert run(lib.msa_rope_write, ks=2.95e-39, qs=2.95e-39) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.95e-39, 1e-38, 1e-20, 0.01, 0.0131, 0.1, 0.25, 1 / 3, 0.7, 1.9999999, 3.0, 1e20, 1e37, 1e38, 3.4e38])
def test_codes_of_q_and_k(scale):
    """Values around the middles of two codes, and all of 16 bits, neither normalised nor rotated.  The reciprocal is off by
    2^-24 of itself (2^-23 where it is no normal number, 2^-128 at least), the product by as much."""
    s32 = float(np.float32(scale))
    codes = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2 * s32
    near = (mid[:, None] * (1 + torch.arange(-40, 41, device="cuda") * 2.0 ** -23)).float()
    every = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.uint16)
    for x in (near.flatten(), every.view(torch.bfloat16), every.view(torch.float16)):
        x = torch.cat([x, -x])
        x = x[~torch.isnan(x)]
        T = -(-x.numel() // 128)
        k = torch.nn.functional.pad(x, (0, T * 128 - x.numel())).view(T, 1, 128)
        pages = T // 128 + 1
        table, cu = torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.tensor([0, T], dtype=torch.int32, device="cuda")
        kv = torch.zeros((pages, 1, 128, 256), dtype=torch.uint8, device="cuda")
        q = msa.msa_rope_write(msa.MsaRope([]), k, k, k, kv, s32, s32, 1.0, table, cu, cu)
        w = k.double() / s32
        lo, hi = (w - w.abs() * 2.0 ** -21, w + w.abs() * 2.0 ** -21)
        lo, hi = (torch.nan_to_num(t, posinf=448, neginf=-448).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() for t in (lo, hi))
        for got in (q.double(), kv.view(torch.float8_e4m3fn).view(-1, 256)[:T, :128].reshape(T, 1, 128).double()):
            assert ((got >= lo) & (got <= hi)).all()
