"""What a server calls around a step of decoding with trees of drafted tokens
(and around any step): rotation with the cache write, tree masks and attention,
acceptance, log probabilities.

Argument marshalling only, as in ``serve.py``, whose checks these calls share;
``include/msa.h`` has each call's meaning.  Tensors have to be on the current
device.

A decode step waits for the host's way to each launch, so the form that it uses
(outputs to be made, the current stream, no status) is checked and called by the
compiled module of ``csrc/binding.cpp``; what that does not take, other forms and
arguments that are not sound, is looked at here one by one, with its messages.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import threading
import warnings

import torch

from . import HEAD_DIM, MsaRopeStruct, _build, load
from .serve import (_E4M3, _F32, _I32, _TYPES, _WORD, _attend, _check, _fail, _handle, _new, _place,
                    _pool, _ptr, _requests, _rows, _status, _table, _tensor)

ROPE_MAX_PAIRS = 64
ROPE_MAX_AXES = 8
TREE_MAX_TOKENS = 256
TREE_MAX_LAYERS = 128
LOGPROBS_MAX_TOP = 32


_binding = None
_binding_lock = threading.Lock()


def load_binding():
    """The compiled module (building it first if it is missing)."""
    global _binding
    with _binding_lock:
        if _binding is not None:
            return _binding
        lib, path = load(), _build.build_binding()
        loader = importlib.machinery.ExtensionFileLoader("msa_binding", path)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location("msa_binding", path, loader=loader))
        loader.exec_module(module)
        module.connect(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.msa_rope_write, lib.msa_rope_write_nvfp4, lib.msa_tree_mask, lib.msa_tree_accept,
            lib.msa_tree_accept_nvfp4, lib.msa_logprobs, lib.msa_tree_attention,
            lib.msa_prefix_attention_workspace_bytes)])
        _binding = module
        return module


class _Checked:
    """In place of the compiled module where there is none: takes no call, so that
    every one goes through the checks here and ctypes, to the same library."""

    rope_write = tree_mask = tree_attention = tree_accept = logprobs = staticmethod(lambda *args: None)


_way = None


def _find_way():
    """What the calls try first: the compiled module, or, where it cannot be built
    (no C++ compiler, no headers), with a warning, none."""
    global _way
    load()
    try:
        _way = load_binding()
    except (RuntimeError, OSError, ImportError) as e:
        warnings.warn("the tree calls take 5-25 us more of the host's time each: their compiled module "
                      "could not be built or loaded: %s" % e, RuntimeWarning, stacklevel=4)
        _way = _Checked
    return _way


def msa_rope_turns(inv_freq):
    """Frequencies in radians a position as fractions of a turn: a list of
    whole numbers in steps of 2^-64 turns."""
    freq = [float(f) for f in inv_freq]
    n = len(freq)
    turns = (ctypes.c_uint64 * max(n, 1))()
    _check(load().msa_rope_turns((ctypes.c_double * max(n, 1))(*freq), n, turns), "msa_rope_turns")
    return list(turns)[:n]


def _whole(x, name):
    """A whole number of any type (no fraction cut off)."""
    try:
        n = int(x)
        if n == x:
            return n
    except (TypeError, ValueError, OverflowError):
        pass
    _fail("%s must be a whole number, got %r", name, x)


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
    or None for none (their values are copied, which waits for the current
    stream), with eps.  It has to live as long as calls and graphs that use it
    run."""

    def __init__(self, inv_freq, interleaved=False, axes=None, q_norm=None, k_norm=None, eps=1e-6):
        freq = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else list(inv_freq)
        if len(freq) > ROPE_MAX_PAIRS:
            _fail("at most %d frequencies, got %d", ROPE_MAX_PAIRS, len(freq))
        axis = [0] * len(freq) if axes is None else [_whole(a, "an axis") for a in axes]
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
        self._address = ctypes.addressof(s)
        weights = [w.get_device() for w in (self.q_norm, self.k_norm) if w is not None]
        if len(set(weights)) > 1:
            _fail("q_norm and k_norm are on different devices")
        self._device = weights[0] if weights else -1
        # the copies are there for calls on any stream (those of a capture on its own)
        if weights and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self._device).synchronize()


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
    if type(rope) is MsaRope and q_out is status is stream is None:
        r = (_way or _find_way()).rope_write(
            rope._address, rope.axes, rope._device, fp4, q, k, v, kv, q_scale, k_scale, v_scale,
            block_table, cu_q, cu_k, positions)
        if r.__class__ is int:
            _check(r, name)
        if r is not None:
            return r
    dev = _check_rope(fp4, rope, q, k, v, kv, q_scale, block_table, cu_q, cu_k, positions, q_out,
                      status)
    T, Hkv, _ = k.shape
    ks, vs, table, handle = k.stride(), v.stride(), block_table.shape, _handle(stream, dev)
    Hq, qs = (0, (0, 0)) if q is None else (q.shape[1], q.stride())
    if q is not None and q_out is None:
        q_out = _new((T, Hq, HEAD_DIM), torch.bfloat16 if q_scale is None else torch.float8_e4m3fn,
                     dev, handle)
    _check(getattr(load(), name)(
        rope._address, _ptr(positions), _ptr(q), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
        v.data_ptr(), vs[0], vs[1], _TYPES[k.dtype], _ptr(q_out), q_scale is None,
        1.0 if q_scale is None else q_scale, kv.data_ptr(), kv.shape[0], k_scale, v_scale,
        block_table.data_ptr(), table[1], cu_q.data_ptr(), cu_k.data_ptr(), table[0], T, Hq, Hkv,
        _ptr(status), handle), name)
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
    n = _whole(max_seqlen_q, "max_seqlen_q")
    if not 0 <= n <= TREE_MAX_TOKENS:
        _fail("max_seqlen_q must be 0 .. %d, got %d", TREE_MAX_TOKENS, n)
    return n


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
    if mask is positions is status is stream is None:
        r = (_way or _find_way()).tree_mask(parents, cu_seqlens_q, cu_seqlens_k,
                                                   max_seqlen_q)
        if r.__class__ is int:
            _check(r, "msa_tree_mask")
        if r is not None:
            return r
    n = _tree_limit(max_seqlen_q)
    words = (n + 31) // 32
    T = parents.shape[0] if parents is not None and parents.dim() == 1 else 0
    _check_tree({"parents": parents}, cu_seqlens_q, cu_seqlens_k,
                {"mask": (mask, _WORD, (T, words)), "positions": (positions, _I32, (T,))}, status)
    dev = _place(parents, cu_seqlens_q, cu_seqlens_k, mask, positions, status)
    _apart({"mask": mask, "positions": positions},
           {"parents": parents, "cu_seqlens_q": cu_seqlens_q, "cu_seqlens_k": cu_seqlens_k})
    handle = _handle(stream, dev)
    mask = _new((T, words), torch.int32, dev, handle) if mask is None else mask
    positions = _new((T,), torch.int32, dev, handle) if positions is None else positions
    _check(load().msa_tree_mask(parents.data_ptr(), cu_seqlens_q.data_ptr(),
                                cu_seqlens_k.data_ptr(), cu_seqlens_q.shape[0] - 1, T, n,
                                mask.data_ptr(), positions.data_ptr(), _ptr(status), handle),
           "msa_tree_mask")
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
    if workspace is out is lse is status is stream is None:
        r = (_way or _find_way()).tree_attention(
            q, kv, q_scale, k_scale, v_scale, softmax_scale, block_table, cu_seqlens_q,
            cu_seqlens_k, mask, prefix_pages, max_seqlen_q, max_seqlen_k, want_lse)
        if r.__class__ is int:
            _check(r, "msa_tree_attention")
        if r is not None:
            return r
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
    if tokens is accepted is path is status is stream is None:
        r = (_way or _find_way()).tree_accept(fp4, drafts, parents, chosen, cu_q, cu_k, max_q,
                                                     kv, table)
        if r.__class__ is int:
            _check(r, name)
        if r is not None:
            return r
    n = _tree_limit(max_q)
    pools = _pools(kv)
    dev = _check_accept(fp4, drafts, parents, chosen, cu_q, cu_k, n, pools, table, tokens, accepted,
                        path, status)
    B, L, handle = cu_q.shape[0] - 1, len(pools), _handle(stream, dev)
    tokens = _new((B, n), torch.int32, dev, handle) if tokens is None else tokens
    accepted = _new((B,), torch.int32, dev, handle) if accepted is None else accepted
    path = _new((B, n), torch.int32, dev, handle) if path is None else path
    at = (ctypes.c_void_p * max(L, 1))(*[p.data_ptr() for p in pools])
    pages, Hkv = pools[0].shape[:2] if L else (0, 0)
    _check(getattr(load(), name)(
        drafts.data_ptr(), parents.data_ptr(), chosen.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
        B, drafts.shape[0], n, ctypes.addressof(at), L, pages, Hkv, table.data_ptr() if L else None,
        table.shape[1] if L else 0, tokens.data_ptr(), accepted.data_ptr(), path.data_ptr(),
        _ptr(status), handle), name)
    return tokens, accepted, path


def msa_tree_accept(draft_tokens, parents, chosen, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                    kv=None, block_table=None, tokens=None, accepted=None, path=None, status=None,
                    stream=None):
    """Which drafted tokens of each request's tree stand, and their rows moved in
    the cache.  draft_tokens, parents, chosen int32 [T]: each node's token, its
    parent (as in msa_tree_mask) and the target's own token after it (the best,
    as msa_logprobs gives it, or a drawn one).  The path starts at a request's
    first token and follows the target's choices; a negative draft stands never.  kv: the pools of all layers,
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
    if logprobs is ranks is entropy is top_tokens is top_logprobs is stream is None:
        r = (_way or _find_way()).logprobs(logits, tokens, top)
        if r.__class__ is int:
            _check(r, "msa_logprobs")
        if r is not None:
            return r
    top = _whole(top, "top")
    if not 0 <= top <= LOGPROBS_MAX_TOP:
        _fail("top must be 0 .. %d, got %d", LOGPROBS_MAX_TOP, top)
    dev = _check_logprobs(logits, tokens, top,
                          {"logprobs": logprobs, "ranks": ranks, "entropy": entropy,
                           "top_tokens": top_tokens, "top_logprobs": top_logprobs})
    T, V = logits.shape
    handle = _handle(stream, dev)

    def new(t, shape, dtype):
        return _new(shape, dtype, dev, handle) if t is None else t

    if tokens is not None:
        logprobs, ranks = new(logprobs, (T,), torch.float32), new(ranks, (T,), torch.int32)
    entropy = new(entropy, (T,), torch.float32)
    top_tokens = new(top_tokens, (T, top), torch.int32)
    top_logprobs = new(top_logprobs, (T, top), torch.float32)
    _check(load().msa_logprobs(
        logits.data_ptr(), logits.stride(0), _TYPES[logits.dtype], _ptr(tokens), T, V, top,
        _ptr(logprobs), _ptr(ranks), entropy.data_ptr(), top_tokens.data_ptr(),
        top_logprobs.data_ptr(), handle), "msa_logprobs")
    return logprobs, ranks, entropy, top_tokens, top_logprobs
