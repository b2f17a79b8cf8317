"""What a server calls around a step of decoding with trees of drafted tokens
(and around any step): rotation with the cache write, tree masks and attention,
acceptance, log probabilities.

Argument marshalling only, as in ``serve.py``, whose way of checking these
calls share; ``include/msa.h`` has each call's meaning.  Tensors have to be on
the current device.
"""
from __future__ import annotations

import ctypes

import torch

from . import HEAD_DIM, MsaError, MsaRopeStruct, load
from .serve import (_E4M3, _I32, _NOT_SOUND, _PAGE, _PAGE4, _TYPES, _check, _fail, _handle, _new,
                    _place, _pool, _ptr, _requests, _rows, _status, _table, _tensor)

ROPE_MAX_PAIRS = 64
ROPE_MAX_AXES = 8


def msa_rope_turns(inv_freq):
    """Frequencies in radians a position as fractions of a turn: a list of
    whole numbers in steps of 2^-64 turns."""
    freq = [float(f) for f in inv_freq]
    n = len(freq)
    turns = (ctypes.c_uint64 * max(n, 1))()
    _check(load().msa_rope_turns((ctypes.c_double * max(n, 1))(*freq), n, turns), "msa_rope_turns")
    return list(turns)[:n]


def _weight(w, name):
    if w is None:
        return None
    if not isinstance(w, torch.Tensor) or tuple(w.shape) != (HEAD_DIM,) or w.dtype not in _TYPES:
        _fail("%s must be a tensor [%d] of one of %s", name, HEAD_DIM, tuple(_TYPES))
    if not w.is_cuda:
        _fail("%s must be a CUDA tensor", name)
    return w.detach().to(torch.float32, copy=True).contiguous()


class MsaRope:
    """How a model rotates (and normalises) its heads, made once: inv_freq,
    the frequency of each rotated pair in radians a position (a sequence or
    tensor of at most 64; scaled ones as a model's context extension gives
    them); interleaved: pair j is values 2j and 2j + 1 of a head, else j and
    j + len(inv_freq); axes: for positions of several axes, the axis of each
    pair; q_norm, k_norm: weights [128] of the heads' root-mean-square norms,
    or None for none (their values are copied), with eps."""

    def __init__(self, inv_freq, interleaved=False, axes=None, q_norm=None, k_norm=None, eps=1e-6):
        freq = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else list(inv_freq)
        if len(freq) > ROPE_MAX_PAIRS:
            _fail("at most %d frequencies, got %d", ROPE_MAX_PAIRS, len(freq))
        axis = [0] * len(freq) if axes is None else [int(a) for a in axes]
        if len(axis) != len(freq) or any(not 0 <= a < ROPE_MAX_AXES for a in axis):
            _fail("axes must be an axis below %d for each of the %d frequencies", ROPE_MAX_AXES,
                  len(freq))
        if not 0 <= float(eps) < 3e38:
            _fail("eps must be finite and not negative")
        self.q_norm, self.k_norm = _weight(q_norm, "q_norm"), _weight(k_norm, "k_norm")
        self.axes = max(axis, default=0) + 1
        s = self._struct = MsaRopeStruct()
        s.pairs, s.interleaved, s.axes, s.eps = len(freq), bool(interleaved), self.axes, float(eps)
        s.q_norm, s.k_norm = _ptr(self.q_norm), _ptr(self.k_norm)
        s.turns[:len(freq)] = msa_rope_turns(freq)
        s.axis[:len(freq)] = axis
        self._at = ctypes.byref(s)


def _reach(t):
    """First and last byte + 1 of a strided tensor."""
    at = t.data_ptr()
    if not t.numel():
        return at, at
    n = sum(s * (d - 1) for s, d in zip(t.stride(), t.shape)) + 1
    return at, at + n * t.element_size()


def _fits(shape, axes, T):
    """Whether positions have a row of T for each axis (further rows are not
    read)."""
    return (len(shape) == 2 and shape[0] >= axes and shape[1] == T) or (axes == 1 and shape == (T,))


def _check_rope(fp4, rope, q, k, v, kv, q_scale, block_table, cu_q, cu_k, positions, q_out, status):
    if not isinstance(rope, MsaRope):
        _fail("rope must be an MsaRope")
    _, Hkv = _pool(kv, fp4)
    B = _requests(cu_q, "cu_seqlens_q")
    _tensor(cu_k, "cu_seqlens_k", _I32, (B + 1,))
    _table(block_table, B)
    if k is None or v is None or k.dim() != 3:
        _fail("k and v must be [T, Hkv, 128]")
    T = k.shape[0]
    _rows(k, "k", (T, Hkv, HEAD_DIM)), _rows(v, "v", (T, Hkv, HEAD_DIM))
    if k.dtype != v.dtype:
        _fail("k and v have different dtypes: %s and %s", k.dtype, v.dtype)
    if q is None:
        if q_out is not None:
            _fail("q_out without q")
    else:
        if q.dim() != 3:
            _fail("q must be [T, Hq, 128], got %s", tuple(q.shape))
        _rows(q, "q", (T, q.shape[1], HEAD_DIM))
        if q.dtype != k.dtype:
            _fail("q and k have different dtypes: %s and %s", q.dtype, k.dtype)
        if q_out is not None:
            _tensor(q_out, "q_out", _E4M3 if q_scale is not None else (torch.bfloat16,),
                    tuple(q.shape))
    if positions is not None:
        _tensor(positions, "positions", _I32)
        if not _fits(positions.shape, rope.axes, T):
            _fail("positions must be [%d, %d]%s, got %s", rope.axes, T,
                  " or [%d]" % T if rope.axes == 1 else "", tuple(positions.shape))
    _status(status)
    dev = _place(kv, k, v, q, block_table, cu_q, cu_k, positions, q_out, status, rope.q_norm,
                 rope.k_norm)
    if q_out is not None:
        lo, hi = _reach(q_out)
        for name, t in (("q", q), ("k", k), ("v", v), ("kv", kv), ("positions", positions),
                        ("block_table", block_table)):
            if t is not None:
                a, b = _reach(t)
                if a < hi and lo < b:
                    _fail("q_out must not share memory with %s", name)
    return dev


def _rope_write(name, fp4, rope, q, k, v, kv, q_scale, k_scale, v_scale, block_table, cu_q, cu_k,
                positions, q_out, status, stream):
    try:
        shape, pool, table, (T, Hq, dim) = k.shape, kv.shape, block_table.shape, q.shape
        ks, vs, qs = k.stride(), v.stride(), q.stride()
        dev = kv.get_device()
        sound = (
            type(rope) is MsaRope and (kv.dtype is torch.uint8 or (kv.dtype in _E4M3 and not fp4))
            and pool[2:] == (_PAGE4 if fp4 else _PAGE) and shape[1:] == (pool[1], HEAD_DIM)
            and len(table) == 2 and cu_q.shape == cu_k.shape == (table[0] + 1,)
            and v.shape == shape and ks[2] == 1 == vs[2] and k.dtype is v.dtype is q.dtype
            and k.dtype in _TYPES and T == shape[0] and dim == HEAD_DIM and qs[2] == 1
            and cu_q.dtype is cu_k.dtype is block_table.dtype is torch.int32
            and (positions is None
                 or (positions.dtype is torch.int32 and positions.is_contiguous()
                     and positions.get_device() == dev
                     and _fits(positions.shape, rope.axes, T)))
            and kv.is_contiguous() and block_table.is_contiguous() and cu_q.is_contiguous()
            and cu_k.is_contiguous() and q_out is None and status is None and dev >= 0
            and (rope.q_norm is None or rope.q_norm.get_device() == dev)
            and (rope.k_norm is None or rope.k_norm.get_device() == dev)
            and dev == k.get_device() == v.get_device() == q.get_device()
            == block_table.get_device() == cu_q.get_device() == cu_k.get_device()
            == torch._C._cuda_getDevice())
    except _NOT_SOUND:
        sound = False
    if not sound:
        dev = _check_rope(fp4, rope, q, k, v, kv, q_scale, block_table, cu_q, cu_k, positions, q_out,
                    status)
    handle = _handle(stream, dev)
    if q is None:
        shape, pool, table = k.shape, kv.shape, block_table.shape
        ks, vs, qs, Hq = k.stride(), v.stride(), (0, 0), 0
    elif q_out is None:
        q_out = _new((T, Hq, HEAD_DIM), torch.bfloat16 if q_scale is None else torch.float8_e4m3fn,
                     dev, handle)
    rc = getattr(load(), name)(
        rope._at, _ptr(positions), _ptr(q), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(),
        vs[0], vs[1], _TYPES[k.dtype], _ptr(q_out), q_scale is None,
        1.0 if q_scale is None else q_scale, kv.data_ptr(), pool[0], k_scale, v_scale,
        block_table.data_ptr(), table[1], cu_q.data_ptr(), cu_k.data_ptr(), table[0], shape[0], Hq,
        pool[1], _ptr(status), handle)
    if rc:
        _check(rc, name)
    return q_out


def msa_rope_write(rope, q, k, v, kv, q_scale, k_scale, v_scale, block_table, cu_seqlens_q,
                   cu_seqlens_k, positions=None, q_out=None, status=None, stream=None):
    """Normalise (where rope has weights) and rotate Q and K, quantise Q for
    the attention, and write K and V into the E4M3 pool kv
    [num_pages, Hkv, 128, 256] as msa_kv_write does.  q [T, Hq, 128] (or None),
    k, v [T, Hkv, 128] in fp32, bf16 or fp16, strided as in msa_kv_write.
    positions: int32 [T], or [axes, T] (rows behind the last axis that rope
    uses are not read); None: the tokens' places in their sequences.  Returns Q as the attention takes it: E4M3 codes of Q / q_scale
    [T, Hq, 128], or bf16 where q_scale is None (for msa_prefill_bf16q).  Rows
    behind cu_seqlens_q's last, and of tokens that status would tell of, keep
    their contents, which in new tensors are undefined.  status as in
    msa_kv_write."""
    return _rope_write("msa_rope_write", False, rope, q, k, v, kv, q_scale, k_scale, v_scale,
                       block_table, cu_seqlens_q, cu_seqlens_k, positions, q_out, status, stream)


def msa_rope_write_nvfp4(rope, q, k, v, kv4, q_scale, k_scale, v_scale, block_table, cu_seqlens_q,
                         cu_seqlens_k, positions=None, q_out=None, status=None, stream=None):
    """msa_rope_write into an NVFP4 pool kv4 uint8 [num_pages, Hkv, 2, 9216],
    as msa_kv_write_nvfp4 writes it."""
    return _rope_write("msa_rope_write_nvfp4", True, rope, q, k, v, kv4, q_scale, k_scale, v_scale,
                       block_table, cu_seqlens_q, cu_seqlens_k, positions, q_out, status, stream)
