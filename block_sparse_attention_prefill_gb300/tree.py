"""What a server calls around a step of decoding with trees of drafted tokens
(and around any step): rotation with the cache write, tree masks and attention,
acceptance, log probabilities.

Argument marshalling only, as in ``serve.py``, whose way of checking these
calls share; ``include/msa.h`` has each call's meaning.  Tensors have to be on
the current device.
"""
from __future__ import annotations

import array
import ctypes
from operator import attrgetter

import torch

from . import HEAD_DIM, MsaRopeStruct, load
from .serve import (_DEVICES, _E4M3, _F32, _I32, _NOT_SOUND, _PAGE, _PAGE4, _TYPES, _WORD, _attend,
                    _check, _fail, _handle, _new, _place, _pool, _ptr, _requests, _rows, _status,
                    _table, _tensor)

# Names that a decode step looks up often.
_int32, _float32, _e4m3, _u8 = torch.int32, torch.float32, torch.float8_e4m3fn, torch.uint8
_empty = torch.empty
_current = getattr(torch._C, "_cuda_getDevice", None)
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_data_ptr, _contiguous, _device = (torch.Tensor.data_ptr, torch.Tensor.is_contiguous,
                                   torch.Tensor.get_device)
_dtype, _shape = attrgetter("dtype"), attrgetter("shape")

ROPE_MAX_PAIRS = 64
ROPE_MAX_AXES = 8
TREE_MAX_TOKENS = 256
TREE_MAX_LAYERS = 128
LOGPROBS_MAX_TOP = 32


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


def _apart(outs, inputs):
    """Refuses outputs that share memory with inputs or with one another (by
    name; None: not there)."""
    reach = [(name, *_reach(t)) for name, t in outs.items() if t is not None]
    rest = [(name, *_reach(t)) for name, t in inputs.items() if t is not None]
    for i, (name, lo, hi) in enumerate(reach):
        for other, a, b in reach[:i] + rest:
            if a < hi and lo < b:
                _fail("%s must not share memory with %s", name, other)


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
    _apart({"q_out": q_out}, {"q": q, "k": k, "v": v, "kv": kv, "positions": positions,
                              "block_table": block_table, "cu_seqlens_q": cu_q,
                              "cu_seqlens_k": cu_k})
    return dev


def _rope_write(name, fp4, rope, q, k, v, kv, q_scale, k_scale, v_scale, block_table, cu_q, cu_k,
                positions, q_out, status, stream):
    dev = -1
    try:
        shape, pool, table, (T, Hq, dim) = k.shape, kv.shape, block_table.shape, q.shape
        ks, vs, qs = k.stride(), v.stride(), q.stride()
        dev, type_, pos = kv.get_device(), k.dtype, positions
        q_norm, k_norm, kv_type = rope.q_norm, rope.k_norm, kv.dtype
        sound = (
            type(rope) is MsaRope and (kv_type is _u8 or (kv_type is _e4m3 and not fp4))
            and pool[2:] == (_PAGE4 if fp4 else _PAGE) and shape == (T, pool[1], dim) == v.shape
            and dim == HEAD_DIM and len(table) == 2
            and cu_q.shape == cu_k.shape == (table[0] + 1,)
            and ks[2] == vs[2] == qs[2] == 1 and type_ in _TYPES
            and type_ is v.dtype is q.dtype and cu_q.dtype is cu_k.dtype is block_table.dtype
            is _int32 and kv.is_contiguous() and block_table.is_contiguous()
            and cu_q.is_contiguous() and cu_k.is_contiguous()
            and (pos is None or (pos.dtype is _int32 and _fits(pos.shape, rope.axes, T)
                                 and pos.is_contiguous() and pos.get_device() == dev))
            and q_out is None and status is None and dev >= 0
            and (q_norm is None or q_norm.get_device() == dev)
            and (k_norm is None or k_norm.get_device() == dev)
            and dev == k.get_device() == v.get_device() == q.get_device()
            == block_table.get_device() == cu_q.get_device() == cu_k.get_device() == _current())
    except _NOT_SOUND:
        sound = False
    if not sound:
        dev = _check_rope(fp4, rope, q, k, v, kv, q_scale, block_table, cu_q, cu_k, positions, q_out,
                          status)
    handle = _raw(dev) if stream is None else _handle(stream, dev)
    if q is None:
        shape, pool, table, type_ = k.shape, kv.shape, block_table.shape, k.dtype
        ks, vs, qs, Hq = k.stride(), v.stride(), (0, 0), 0
    elif q_out is None:
        out = torch.bfloat16 if q_scale is None else _e4m3
        q_out = (_empty((T, Hq, HEAD_DIM), dtype=out, device=_DEVICES[dev]) if stream is None
                 else _new((T, Hq, HEAD_DIM), out, dev, handle))
    lib = load()
    rc = (lib.msa_rope_write_nvfp4 if fp4 else lib.msa_rope_write)(
        rope._at, None if positions is None else positions.data_ptr(),
        None if q is None else q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(),
        vs[0], vs[1], _TYPES[type_], None if q is None else q_out.data_ptr(), q_scale is None,
        1.0 if q_scale is None else q_scale, kv.data_ptr(), pool[0], k_scale, v_scale,
        block_table.data_ptr(), table[1], cu_q.data_ptr(), cu_k.data_ptr(), table[0], shape[0], Hq,
        pool[1], None if status is None else status.data_ptr(), handle)
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


def _check_tree(flat, cu_q, cu_k, outs, status):
    """Tensors [T] by name, the lengths, and the outputs' types and shapes."""
    B = _requests(cu_q, "cu_seqlens_q")
    _tensor(cu_k, "cu_seqlens_k", _I32, (B + 1,))
    first = None
    for name, t in flat.items():
        _tensor(t, name, _I32, first)
        if first is None:
            if t.dim() != 1:
                _fail("%s must be [T], got %s", name, tuple(t.shape))
            first = t.shape
    for name, (t, dtypes, shape) in outs.items():
        if t is not None:
            _tensor(t, name, dtypes, shape)
    _status(status)


def _tree_limit(max_seqlen_q):
    if not 0 <= max_seqlen_q <= TREE_MAX_TOKENS:
        _fail("max_seqlen_q must be 0 .. %d, got %d", TREE_MAX_TOKENS, max_seqlen_q)
    return int(max_seqlen_q)


def msa_tree_mask(parents, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, mask=None, positions=None,
                  status=None, stream=None):
    """Ancestor masks and positions of a batch's trees of drafted tokens.
    parents int32 [T]: each token's parent by its place among its request's
    new tokens (at most max_seqlen_q <= 256), parents first, -1 for a root.
    Returns (mask int32 [T, ceil(max_seqlen_q / 32)], positions int32 [T]) for
    msa_tree_attention and msa_rope_write; rows behind cu_seqlens_q's last and
    of requests whose lengths do not fit keep their contents, which in new
    tensors are undefined.  status: an int32 [1] tensor that MSA_STATUS_* bits
    are OR-ed into; without it nothing tells of lengths that do not fit or of
    parents that are no earlier tokens (taken for -1)."""
    n = _tree_limit(max_seqlen_q)
    words = (n + 31) // 32
    try:
        (T,), (B1,), dev = parents.shape, cu_seqlens_q.shape, parents.get_device()
        sound = (
            parents.dtype is cu_seqlens_q.dtype is cu_seqlens_k.dtype is _int32 and B1 > 0
            and cu_seqlens_k.shape == (B1,) and parents.is_contiguous()
            and cu_seqlens_q.is_contiguous() and cu_seqlens_k.is_contiguous()
            and mask is None and positions is None and status is None and dev >= 0
            and dev == cu_seqlens_q.get_device() == cu_seqlens_k.get_device() == _current())
    except _NOT_SOUND:
        sound = False
    if not sound:
        _check_tree({"parents": parents}, cu_seqlens_q, cu_seqlens_k,
                    {"mask": (mask, _WORD, (T, words)), "positions": (positions, _I32, (T,))}
                    if parents is not None and parents.dim() == 1 else {}, status)
        dev = _place(parents, cu_seqlens_q, cu_seqlens_k, mask, positions, status)
        _apart({"mask": mask, "positions": positions},
               {"parents": parents, "cu_seqlens_q": cu_seqlens_q, "cu_seqlens_k": cu_seqlens_k})
    if stream is None:
        handle, on = _raw(dev), _DEVICES[dev]
        if mask is None:
            mask = _empty((T, words), dtype=_int32, device=on)
        if positions is None:
            positions = _empty((T,), dtype=_int32, device=on)
    else:
        handle = _handle(stream, dev)
        if mask is None:
            mask = _new((T, words), _int32, dev, handle)
        if positions is None:
            positions = _new((T,), _int32, dev, handle)
    rc = load().msa_tree_mask(parents.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                              B1 - 1, T, n, mask.data_ptr(), positions.data_ptr(),
                              None if status is None else status.data_ptr(), handle)
    if rc:
        _check(rc, "msa_tree_mask")
    return mask, positions


def msa_tree_attention(q, kv, q_scale, k_scale, v_scale, softmax_scale, block_table, cu_seqlens_q,
                       cu_seqlens_k, mask, prefix_pages, max_seqlen_q, max_seqlen_k,
                       workspace=None, out=None, lse=None, want_lse=True, status=None,
                       stream=None):
    """Dense attention of trees of drafted tokens over the E4M3 pool: as
    msa_prefix_attention (whose arguments, workspace and returns these are),
    with each token attending to all keys before its request's new ones, and of
    these to those whose bits are set in its words of mask, int32 [T, at least
    ceil(max_seqlen_q / 32)] (msa_tree_mask's, or any others); max_seqlen_q at
    most 256.  A token that sees no key gets zeros and lse -inf."""
    n = _tree_limit(max_seqlen_q)
    _tensor(mask, "mask", _WORD)
    shape = mask.shape
    if q is None or q.dim() != 3 or len(shape) != 2 or shape[0] != q.shape[0] or shape[1] * 32 < n:
        _fail("mask must be [%s, %d or more], got %s",
              "T" if q is None or q.dim() != 3 else q.shape[0], (n + 31) // 32, tuple(shape))
    return _attend("msa_tree_attention", q, kv, q_scale, k_scale, v_scale, softmax_scale,
                   block_table, cu_seqlens_q, cu_seqlens_k, mask, prefix_pages, max_seqlen_q,
                   max_seqlen_k, workspace, out, lse, want_lse, status, stream)


def _pools(kv):
    """The layers' pools of a call, as a list of tensors of one shape."""
    if kv is None:
        return []
    if isinstance(kv, torch.Tensor):
        return list(kv.unbind(0)) if kv.dim() == 5 else [kv]
    return list(kv)


def _check_accept(fp4, drafts, parents, chosen, cu_q, cu_k, n, pools, table, tokens, accepted,
                  path, status):
    B = _requests(cu_q, "cu_seqlens_q")
    _check_tree({"draft_tokens": drafts, "parents": parents, "chosen": chosen}, cu_q, cu_k,
                {"tokens": (tokens, _I32, (B, n)), "accepted": (accepted, _I32, (B,)),
                 "path": (path, _I32, (B, n))}, status)
    if len(pools) > TREE_MAX_LAYERS:
        _fail("at most %d layers, got %d", TREE_MAX_LAYERS, len(pools))
    for p in pools:
        _pool(p, fp4)
        if p.shape != pools[0].shape:
            _fail("the layers' pools differ: %s and %s", tuple(pools[0].shape), tuple(p.shape))
    if pools:
        _table(table, B)
    dev = _place(drafts, parents, chosen, cu_q, cu_k, tokens, accepted, path, status, *pools,
                 table if pools else None)
    spans = sorted(_reach(p) for p in pools)
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        _fail("the layers' pools must not share memory")
    _apart({"tokens": tokens, "accepted": accepted, "path": path},
           {"draft_tokens": drafts, "parents": parents, "chosen": chosen, "cu_seqlens_q": cu_q,
            "cu_seqlens_k": cu_k})
    return dev


def _accept(name, fp4, drafts, parents, chosen, cu_q, cu_k, max_q, kv, table, tokens, accepted,
            path, status, stream):
    n = _tree_limit(max_q)
    pools = _pools(kv)
    L, dev, shape, at = len(pools), -1, (0, 0), None
    try:
        (T,), (B1,), dev = drafts.shape, cu_q.shape, drafts.get_device()
        sound = (
            drafts.dtype is parents.dtype is chosen.dtype is cu_q.dtype is cu_k.dtype is _int32
            and B1 > 0 and parents.shape == chosen.shape == (T,) and cu_k.shape == (B1,)
            and drafts.is_contiguous() and parents.is_contiguous() and chosen.is_contiguous()
            and cu_q.is_contiguous() and cu_k.is_contiguous() and L <= TREE_MAX_LAYERS
            and tokens is None and accepted is None and path is None and status is None
            and dev >= 0 and dev == parents.get_device() == chosen.get_device()
            == cu_q.get_device() == cu_k.get_device() == _current())
        if sound and L:
            # all pools alike: what they have in common is looked at once
            (shape,), (type_,), (on,) = (set(map(_shape, pools)), set(map(_dtype, pools)),
                                         set(map(_device, pools)))
            sound = (
                shape[2:] == (_PAGE4 if fp4 else _PAGE) and len(shape) == 4 and on == dev
                and (type_ is _u8 or (type_ is _e4m3 and not fp4))
                and all(map(_contiguous, pools)) and table.dtype is _int32 and table.dim() == 2
                and table.shape[0] == B1 - 1 and table.is_contiguous()
                and table.get_device() == dev)
    except _NOT_SOUND:
        sound = False
    if not sound:
        dev = _check_accept(fp4, drafts, parents, chosen, cu_q, cu_k, n, pools, table, tokens,
                            accepted, path, status)
        shape = pools[0].shape if L else shape
    B = B1 - 1
    if stream is None:
        handle, on = _raw(dev), _DEVICES[dev]
        if tokens is None:
            tokens = _empty((B, n), dtype=_int32, device=on)
        if accepted is None:
            accepted = _empty((B,), dtype=_int32, device=on)
        if path is None:
            path = _empty((B, n), dtype=_int32, device=on)
    else:
        handle = _handle(stream, dev)
        tokens = _new((B, n), _int32, dev, handle) if tokens is None else tokens
        accepted = _new((B,), _int32, dev, handle) if accepted is None else accepted
        path = _new((B, n), _int32, dev, handle) if path is None else path
    if L:
        at = array.array("Q", map(_data_ptr, pools))  # (kept until the call has read it)
    lib = load()
    rc = (lib.msa_tree_accept_nvfp4 if fp4 else lib.msa_tree_accept)(
        drafts.data_ptr(), parents.data_ptr(), chosen.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
        B, T, n, at.buffer_info()[0] if L else None, L, shape[0], shape[1],
        table.data_ptr() if L else None, table.shape[1] if L else 0, tokens.data_ptr(),
        accepted.data_ptr(), path.data_ptr(), None if status is None else status.data_ptr(), handle)
    if rc:
        _check(rc, name)
    return tokens, accepted, path


def msa_tree_accept(draft_tokens, parents, chosen, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                    kv=None, block_table=None, tokens=None, accepted=None, path=None, status=None,
                    stream=None):
    """Which drafted tokens of each request's tree stand, and their rows moved in
    the cache.  draft_tokens, parents, chosen int32 [T]: each node's token, its
    parent (as in msa_tree_mask) and the target's own token after it (the best,
    as msa_logprobs gives it, or a drawn one).  The path starts at a request's
    first token and follows the target's choices.  kv: the pools of all layers,
    a sequence of E4M3 pools [num_pages, Hkv, 128, 256] (at most 128, which
    share no memory), one pool, a tensor [layers, ...] of them, or None: the
    rows of the path are moved to follow the context directly, so that the
    sequence goes on at length seq_len - q_len + 1 + accepted.  Returns (tokens
    int32 [B, max_seqlen_q]: the drafts that stand, the next token, -1; accepted
    int32 [B]; path int32 [B, max_seqlen_q]: the nodes, the first with them,
    then -1).  status as in msa_tree_mask."""
    return _accept("msa_tree_accept", False, draft_tokens, parents, chosen, cu_seqlens_q,
                   cu_seqlens_k, max_seqlen_q, kv, block_table, tokens, accepted, path, status,
                   stream)


def msa_tree_accept_nvfp4(draft_tokens, parents, chosen, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                          kv=None, block_table=None, tokens=None, accepted=None, path=None,
                          status=None, stream=None):
    """msa_tree_accept with NVFP4 pools uint8 [num_pages, Hkv, 2, 9216]."""
    return _accept("msa_tree_accept_nvfp4", True, draft_tokens, parents, chosen, cu_seqlens_q,
                   cu_seqlens_k, max_seqlen_q, kv, block_table, tokens, accepted, path, status,
                   stream)


def _check_logprobs(logits, tokens, top, outs):
    _tensor(logits, "logits", _TYPES, None, False)
    if logits.dim() != 2:
        _fail("logits must be [T, V], got %s", tuple(logits.shape))
    T, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        _fail("logits' rows must be contiguous")
    if tokens is not None:
        _tensor(tokens, "tokens", _I32, (T,))
    elif outs["logprobs"] is not None or outs["ranks"] is not None:
        _fail("logprobs and ranks need tokens")
    for name, dtypes, shape in (("logprobs", _F32, (T,)), ("ranks", _I32, (T,)),
                                ("entropy", _F32, (T,)), ("top_tokens", _I32, (T, top)),
                                ("top_logprobs", _F32, (T, top))):
        if outs[name] is not None:
            _tensor(outs[name], name, dtypes, shape)
    dev = _place(logits, tokens, *outs.values())
    _apart(outs, {"logits": logits, "tokens": tokens})
    return dev


def msa_logprobs(logits, tokens=None, top=0, logprobs=None, ranks=None, entropy=None,
                 top_tokens=None, top_logprobs=None, stream=None):
    """Log probabilities from logits [T, V] (fp32, bf16 or fp16; rows may be
    strided; -inf: a probability of 0) of the given tokens int32 [T], with their
    ranks, and each row's entropy and best alternatives (top <= 32).  Returns
    (logprobs fp32 [T], ranks int32 [T] (0: the best), entropy fp32 [T] in nats,
    top_tokens int32 [T, top], top_logprobs fp32 [T, top]); the first two are
    None without tokens.  Of equal logits the lower index comes first.  A token
    outside [0, V) has -inf and rank -1; a row with a NaN has NaN, but for the
    tokens and ranks."""
    if not 0 <= top <= LOGPROBS_MAX_TOP:
        _fail("top must be 0 .. %d, got %d", LOGPROBS_MAX_TOP, top)
    dev = -1
    try:
        (T, V), (row, one), dev, type_ = (logits.shape, logits.stride(), logits.get_device(),
                                          logits.dtype)
        sound = (
            type_ in _TYPES and (one == 1 or V == 1)
            and (tokens is None or (tokens.dtype is _int32 and tokens.shape == (T,)
                                    and tokens.is_contiguous() and tokens.get_device() == dev))
            and logprobs is None and ranks is None and entropy is None and top_tokens is None
            and top_logprobs is None and dev >= 0 and dev == _current())
    except _NOT_SOUND:
        sound = False
    if not sound:
        dev = _check_logprobs(logits, tokens, top,
                              {"logprobs": logprobs, "ranks": ranks, "entropy": entropy,
                               "top_tokens": top_tokens, "top_logprobs": top_logprobs})
    given = tokens is not None
    if stream is None and sound:
        handle, on = _raw(dev), _DEVICES[dev]
        if given:
            logprobs = _empty((T,), dtype=_float32, device=on)
            ranks = _empty((T,), dtype=_int32, device=on)
        entropy = _empty((T,), dtype=_float32, device=on)
        top_tokens = _empty((T, top), dtype=_int32, device=on)
        top_logprobs = _empty((T, top), dtype=_float32, device=on)
    else:
        handle = _handle(stream, dev)
        if given and logprobs is None:
            logprobs = _new((T,), _float32, dev, handle)
        if given and ranks is None:
            ranks = _new((T,), _int32, dev, handle)
        if entropy is None:
            entropy = _new((T,), _float32, dev, handle)
        if top_tokens is None:
            top_tokens = _new((T, top), _int32, dev, handle)
        if top_logprobs is None:
            top_logprobs = _new((T, top), _float32, dev, handle)
    rc = load().msa_logprobs(
        logits.data_ptr(), row, _TYPES[type_], tokens.data_ptr() if given else None, T, V, top,
        logprobs.data_ptr() if given else None, ranks.data_ptr() if given else None,
        entropy.data_ptr(), top_tokens.data_ptr(), top_logprobs.data_ptr(), handle)
    if rc:
        _check(rc, "msa_logprobs")
    return logprobs, ranks, entropy, top_tokens, top_logprobs
