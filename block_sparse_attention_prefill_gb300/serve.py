"""What a server calls around the block-sparse attention: cache writes and
reads, dense attention behind a shared prefix, draft verification.

Argument marshalling only, as in the package's ``__init__`` (whose public
names these are); ``include/msa.h`` has each call's meaning.  These calls
check every shape, type, stride and device here, because the library sees
only pointers; tensors have to be on the current device.

A decode step waits for these checks, so each call first looks whether all of
them hold in one expression (about half the time of the checks one by one),
and goes through them one by one, with their messages, only where not.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import (DTYPE_BF16, DTYPE_F16, DTYPE_F32, HEAD_DIM, MsaError, NVFP4_SLOT_BYTES, PAGE_SIZE,
               _empty, load, status_string)

# What the checks below raise on a sound call's shortcut for what is not a
# tensor or has other dimensions.
_NOT_SOUND = (AttributeError, TypeError, ValueError)

_TYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_WORD = (torch.int32, torch.uint32)
_PAGE, _PAGE4 = (PAGE_SIZE, 2 * HEAD_DIM), (2, NVFP4_SLOT_BYTES)


def _fail(what, *args):
    raise MsaError(what % args)


def _check(rc, what):
    if rc:
        raise MsaError("%s: %s (code %d)" % (what, status_string(rc), rc))


def _tensor(t, name, dtypes, shape=None, contiguous=True):
    """Type and shape of a required tensor."""
    if t is None:
        _fail("%s is required", name)
    if t.dtype not in dtypes:
        _fail("%s has dtype %s, expected one of %s", name, t.dtype, dtypes)
    if shape is not None and t.shape != shape:
        _fail("%s must be %s, got %s", name, list(shape), tuple(t.shape))
    if contiguous and not t.is_contiguous():
        _fail("%s must be contiguous", name)


def _place(first, *others):
    """The index of the device that all given tensors share, which must be the
    current one."""
    dev = first.get_device()
    if dev < 0:
        _fail("tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != dev:
            _fail("tensors are on different devices: %s and %s", first.device, t.device)
    if dev != torch._C._cuda_getDevice():
        _fail("tensors are on cuda:%d, the current device is cuda:%d", dev,
              torch.cuda.current_device())
    return dev


def _handle(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


_DEVICES = [torch.device("cuda", i) for i in range(64)]


def _new(shape, dtype, dev, handle):
    """A tensor on device `dev` for use on the stream `handle`, whichever
    stream is current."""
    if handle != torch._C._cuda_getCurrentRawStream(dev):
        return _empty(shape, dtype, _DEVICES[dev], handle)
    return torch.empty(shape, dtype=dtype, device=_DEVICES[dev])


def _ptr(t):
    return None if t is None else t.data_ptr()


def _pool(kv, fp4):
    """(num_pages, Hkv) of a page pool."""
    if fp4:
        _tensor(kv, "kv4", (torch.uint8,))
        shape = kv.shape
        if len(shape) != 4 or shape[2] != 2 or shape[3] != NVFP4_SLOT_BYTES:
            _fail("kv4 must be [any, any, 2, %d], got %s", NVFP4_SLOT_BYTES, tuple(shape))
    else:
        _tensor(kv, "kv", _E4M3)
        shape = kv.shape
        if len(shape) != 4 or shape[2] != PAGE_SIZE or shape[3] != 2 * HEAD_DIM:
            _fail("kv must be [any, any, 128, 256], got %s", tuple(shape))
    return shape[0], shape[1]


def _rows(t, name, shape):
    """Strides of K or V rows [T, Hkv, 128] whose 128 values are contiguous."""
    _tensor(t, name, _TYPES, shape, False)
    token, head, one = t.stride()
    if one != 1:
        _fail("%s must have its 128 values contiguous", name)
    return token, head


def _table(block_table, B):
    _tensor(block_table, "block_table", _I32)
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != B:
        _fail("block_table must be [%d, any], got %s", B, tuple(shape))
    return shape[1]


def _requests(cu, name):
    """B of prefix sums [B + 1]."""
    _tensor(cu, name, _I32)
    if cu.dim() != 1 or cu.shape[0] < 1:
        _fail("%s must be one-dimensional with at least one element", name)
    return cu.shape[0] - 1


def _status(status):
    if status is not None:
        _tensor(status, "status", _WORD, (1,))


def _check_write(fp4, k, v, kv, block_table, cu_q, cu_k, status):
    _, Hkv = _pool(kv, fp4)
    B = _requests(cu_q, "cu_seqlens_q")
    _tensor(cu_k, "cu_seqlens_k", _I32, (B + 1,))
    _table(block_table, B)
    if k is None or v is None or k.dim() != 3:
        _fail("k and v must be [T, Hkv, 128]")
    shape = (k.shape[0], Hkv, HEAD_DIM)
    _rows(k, "k", shape), _rows(v, "v", shape)
    if k.dtype != v.dtype:
        _fail("k and v have different dtypes: %s and %s", k.dtype, v.dtype)
    _status(status)
    _place(kv, k, v, block_table, cu_q, cu_k, status)


def _write(name, fp4, k, v, kv, k_scale, v_scale, block_table, cu_q, cu_k, status, stream):
    try:
        shape, pool, table = k.shape, kv.shape, block_table.shape
        ks, vs = k.stride(), v.stride()
        dev = kv.get_device()
        sound = (
            (kv.dtype is torch.uint8 or (kv.dtype in _E4M3 and not fp4))
            and pool[2:] == (_PAGE4 if fp4 else _PAGE) and shape[1:] == (pool[1], HEAD_DIM)
            and len(table) == 2 and cu_q.shape == cu_k.shape == (table[0] + 1,)
            and v.shape == shape and ks[2] == 1 == vs[2] and k.dtype is v.dtype
            and k.dtype in _TYPES and cu_q.dtype is cu_k.dtype is block_table.dtype is torch.int32
            and kv.is_contiguous() and block_table.is_contiguous() and cu_q.is_contiguous()
            and cu_k.is_contiguous() and status is None and dev >= 0
            and dev == k.get_device() == v.get_device() == block_table.get_device()
            == cu_q.get_device() == cu_k.get_device() == torch._C._cuda_getDevice())
    except _NOT_SOUND:
        sound = False
    if not sound:
        _check_write(fp4, k, v, kv, block_table, cu_q, cu_k, status)
    rc = getattr(load(), name)(
        k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], _TYPES[k.dtype], kv.data_ptr(),
        pool[0], k_scale, v_scale, block_table.data_ptr(), table[1], cu_q.data_ptr(),
        cu_k.data_ptr(), table[0], shape[0], pool[1], _ptr(status), _handle(stream, dev))
    if rc:
        _check(rc, name)


def msa_kv_write(k, v, kv, k_scale, v_scale, block_table, cu_seqlens_q, cu_seqlens_k,
                 status=None, stream=None):
    """Write new tokens into the E4M3 pool kv [num_pages, Hkv, 128, 256].
    k, v [T, Hkv, 128] in fp32, bf16 or fp16 (any token and head strides that
    keep rows on 16 bytes); they are the last q_len positions of each request,
    as in msa_plan.  Rows behind cu_seqlens_q's last are left out.  status: an
    int32 [1] tensor that MSA_STATUS_* bits are OR-ed into; tokens that it
    would tell of are not written, with it or without."""
    _write("msa_kv_write", False, k, v, kv, k_scale, v_scale, block_table, cu_seqlens_q,
           cu_seqlens_k, status, stream)


def msa_kv_write_nvfp4(k, v, kv4, k_scale, v_scale, block_table, cu_seqlens_q, cu_seqlens_k,
                       status=None, stream=None):
    """msa_kv_write into an NVFP4 pool kv4 uint8 [num_pages, Hkv, 2, 9216];
    k_scale / v_scale are the global scales (amax / 448 keeps every block
    scale in range)."""
    _write("msa_kv_write_nvfp4", True, k, v, kv4, k_scale, v_scale, block_table, cu_seqlens_q,
           cu_seqlens_k, status, stream)


def _apart_rows(t, name):
    """Refuses rows [T, Hkv, 128] of an output that share elements (the larger
    stride has to step over all rows of the smaller)."""
    (T, H, _), (token, head, _) = t.shape, t.stride()
    reach = HEAD_DIM
    for stride, n in sorted(((token, T), (head, H))):
        if n > 1 and stride < reach:
            _fail("rows of %s must not overlap", name)
        if n > 1:
            reach += stride * (n - 1)


def _check_read(fp4, kv, block_table, cu, T, starts, k, v, status):
    _, Hkv = _pool(kv, fp4)
    B = _requests(cu, "cu_tokens")
    _table(block_table, B)
    if starts is not None:
        _tensor(starts, "starts", _I32, (B,))
    _status(status)
    if (k is None) != (v is None):
        _fail("give both of k and v, or neither")
    if k is not None:
        for t, name in ((k, "k"), (v, "v")):
            _rows(t, name, (T, Hkv, HEAD_DIM))
            _apart_rows(t, name)
        if k.dtype != v.dtype:
            _fail("k and v have different dtypes: %s and %s", k.dtype, v.dtype)
        if T > 0 and k.data_ptr() == v.data_ptr():
            _fail("k and v must not share rows")
    _place(kv, block_table, cu, starts, k, v, status)


def _read(name, fp4, kv, k_scale, v_scale, block_table, cu, T, starts, dtype, k, v, status,
          stream):
    try:
        pool, table = kv.shape, block_table.shape
        dev = kv.get_device()
        sound = (
            (kv.dtype is torch.uint8 or (kv.dtype in _E4M3 and not fp4))
            and pool[2:] == (_PAGE4 if fp4 else _PAGE)
            and len(table) == 2 and cu.shape == (table[0] + 1,)
            and cu.dtype is block_table.dtype is torch.int32
            and kv.is_contiguous() and block_table.is_contiguous() and cu.is_contiguous()
            and (starts is None or (starts.dtype is torch.int32 and starts.shape == (table[0],)
                                    and starts.is_contiguous() and starts.get_device() == dev))
            and k is None and v is None and status is None and dev >= 0
            and dev == block_table.get_device() == cu.get_device() == torch._C._cuda_getDevice())
    except _NOT_SOUND:
        sound = False
    T = int(T)
    if T < 0:
        _fail("total_tokens must not be negative")
    if not sound:
        _check_read(fp4, kv, block_table, cu, T, starts, k, v, status)
    handle = _handle(stream, dev)
    if k is None:
        shape = (T, pool[1], HEAD_DIM)
        if dtype not in _TYPES:
            _fail("dtype must be one of %s", tuple(_TYPES))
        k, v = _new(shape, dtype, dev, handle), _new(shape, dtype, dev, handle)
        ks = vs = (pool[1] * HEAD_DIM, HEAD_DIM)
    else:
        ks, vs = k.stride(), v.stride()
    rc = getattr(load(), name)(kv.data_ptr(), pool[0], k_scale, v_scale, block_table.data_ptr(),
                               table[1], cu.data_ptr(), _ptr(starts), table[0], T, pool[1],
                               k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                               _TYPES[k.dtype], _ptr(status), handle)
    if rc:
        _check(rc, name)
    return k, v


def msa_kv_read(kv, k_scale, v_scale, block_table, cu_tokens, total_tokens, starts=None,
                dtype=torch.bfloat16, k=None, v=None, status=None, stream=None):
    """Read cached tokens back from an E4M3 pool, dequantised: request b's
    positions starts[b] .. (0 without starts) become rows cu_tokens[b] ..
    cu_tokens[b + 1] - 1 of k and v [total_tokens, Hkv, 128].  k and v may be
    given (any of the three types, strided); rows behind cu_tokens' last, and
    rows whose page is not valid, keep their contents, which in new tensors
    are undefined.  status as in msa_kv_write.  Returns (k, v)."""
    return _read("msa_kv_read", False, kv, k_scale, v_scale, block_table, cu_tokens,
                 total_tokens, starts, dtype, k, v, status, stream)


def msa_kv_read_nvfp4(kv4, k_scale, v_scale, block_table, cu_tokens, total_tokens, starts=None,
                      dtype=torch.bfloat16, k=None, v=None, status=None, stream=None):
    """msa_kv_read from an NVFP4 pool: E4M3(code x block scale) x the global
    scale, what the NVFP4 attention reads."""
    return _read("msa_kv_read_nvfp4", True, kv4, k_scale, v_scale, block_table, cu_tokens,
                 total_tokens, starts, dtype, k, v, status, stream)


def prefix_attention_workspace_bytes(B, T, Hq, Hkv, prefix_pages, max_seqlen_q,
                                     max_seqlen_k) -> int:
    n = ctypes.c_size_t()
    _check(load().msa_prefix_attention_workspace_bytes(B, T, Hq, Hkv, prefix_pages, max_seqlen_q,
                                                       max_seqlen_k, ctypes.byref(n)),
           "msa_prefix_attention_workspace_bytes")
    return n.value


@functools.lru_cache(maxsize=64)
def _attention_bytes(dev, B, T, Hq, Hkv, prefix_pages, max_q, max_k):
    """The same for the current device, `dev`; the size depends on these
    numbers and the device alone, and a decode loop asks for the same one again
    and again."""
    return prefix_attention_workspace_bytes(B, T, Hq, Hkv, prefix_pages, max_q, max_k)


def _check_attention(q, kv, block_table, cu_q, cu_k, workspace, out, lse, status):
    _pool(kv, False)
    _tensor(q, "q", _E4M3)
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        _fail("q must be [any, any, 128], got %s", tuple(q.shape))
    B = _requests(cu_q, "cu_seqlens_q")
    _tensor(cu_k, "cu_seqlens_k", _I32, (B + 1,))
    _table(block_table, B)
    _status(status)
    if out is not None:
        _tensor(out, "out", (torch.bfloat16,), tuple(q.shape))
    if lse is not None:
        _tensor(lse, "lse", _F32, tuple(q.shape[:2]))
    if workspace is not None:
        _tensor(workspace, "workspace", (torch.uint8,))


def msa_prefix_attention(q, kv, q_scale, k_scale, v_scale, softmax_scale, block_table,
                         cu_seqlens_q, cu_seqlens_k, prefix_pages, max_seqlen_q, max_seqlen_k,
                         workspace=None, out=None, lse=None, want_lse=True, status=None,
                         stream=None):
    """Dense causal attention over the E4M3 pool for a batch whose requests
    share their first prefix_pages pages, whose part is computed once for all
    (0: nothing shared).  q E4M3 [T, Hq, 128]; lengths as in msa_plan, all
    queries behind the shared pages.  status: an int32 [1] tensor that
    MSA_STATUS_* bits are OR-ed into; without it nothing tells of lengths that
    do not fit (all rows 0) or entries that are no pages (left out).  Rows
    behind cu_seqlens_q's last keep their contents, which in new tensors are
    undefined.  Returns (out bf16 [T, Hq, 128], lse fp32 [T, Hq] or None)."""
    try:
        pool, table, (T, Hq, dim) = kv.shape, block_table.shape, q.shape
        dev = kv.get_device()
        sound = (
            kv.dtype in _E4M3 and q.dtype in _E4M3 and pool[2:] == _PAGE and dim == HEAD_DIM
            and len(table) == 2 and cu_seqlens_q.shape == cu_seqlens_k.shape == (table[0] + 1,)
            and cu_seqlens_q.dtype is cu_seqlens_k.dtype is block_table.dtype is torch.int32
            and kv.is_contiguous() and q.is_contiguous() and block_table.is_contiguous()
            and cu_seqlens_q.is_contiguous() and cu_seqlens_k.is_contiguous()
            and out is None and lse is None and workspace is None and status is None and dev >= 0
            and dev == q.get_device() == block_table.get_device() == cu_seqlens_q.get_device()
            == cu_seqlens_k.get_device() == torch._C._cuda_getDevice())
    except _NOT_SOUND:
        sound = False
    if not sound:
        _check_attention(q, kv, block_table, cu_seqlens_q, cu_seqlens_k, workspace, out, lse,
                         status)
    B, Hkv = table[0], pool[1]
    # the library answers for the current device: nothing is kept for another,
    # which is refused below
    here = sound or (dev >= 0 and dev == torch._C._cuda_getDevice())
    sizes = (B, T, Hq, Hkv, prefix_pages, max_seqlen_q, max_seqlen_k)
    need = _attention_bytes(dev, *sizes) if here else prefix_attention_workspace_bytes(*sizes)
    if workspace is not None and workspace.numel() < need:
        _fail("workspace too small: %d < %d bytes", workspace.numel(), need)
    if not sound:
        _place(q, kv, block_table, cu_seqlens_q, cu_seqlens_k, workspace, out, lse, status)
    handle = _handle(stream, dev)
    if workspace is None:
        workspace = _new(need, torch.uint8, dev, handle)
    if out is None:
        out = _new((T, Hq, HEAD_DIM), torch.bfloat16, dev, handle)
    if lse is None and want_lse:
        lse = _new((T, Hq), torch.float32, dev, handle)
    rc = load().msa_prefix_attention(
        q.data_ptr(), kv.data_ptr(), pool[0], q_scale, k_scale, v_scale, softmax_scale,
        block_table.data_ptr(), table[1], cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, T,
        Hq, Hkv, prefix_pages, max_seqlen_q, max_seqlen_k, workspace.data_ptr(),
        workspace.numel(), out.data_ptr(), _ptr(lse), _ptr(status), handle)
    if rc:
        _check(rc, "msa_prefix_attention")
    return out, lse


def _probs(t, name, dtypes):
    """Shape of rows [B, n, V] whose values are contiguous."""
    _tensor(t, name, dtypes, None, False)
    shape = t.shape
    if len(shape) != 3:
        _fail("%s must be [any, any, any], got %s", name, tuple(shape))
    if t.stride(2) != 1 and shape[2] > 1:
        _fail("%s's rows must be contiguous", name)
    return shape


def _apart(out, name, inputs):
    """Refuses an output that shares memory with one of the inputs, all
    contiguous, by their names."""
    if out is None:
        return
    at, n = out.data_ptr(), out.numel() * out.element_size()
    for other, t in inputs.items():
        if t is not None and at < t.data_ptr() + t.numel() * t.element_size() and \
                t.data_ptr() < at + n:
            _fail("%s must not share memory with %s", name, other)


def _check_verify(greedy, target, drafts, uniforms, draft_probs, counts, tokens, accepted):
    B, n, V = _probs(target, "target", _TYPES)
    if n < 1:
        _fail("target must have at least one row a request")
    _tensor(drafts, "draft_tokens", _I32, (B, n - 1))
    if not greedy:
        _tensor(uniforms, "uniforms", _F32, (B, n))
    if draft_probs is not None:
        shape = _probs(draft_probs, "draft_probs", (target.dtype,))
        if shape != (B, n - 1, V):
            _fail("draft_probs must be %s, got %s", [B, n - 1, V], tuple(shape))
    if counts is not None:
        _tensor(counts, "num_drafts", _I32, (B,))
    if tokens is not None:
        _tensor(tokens, "tokens", _I32, (B, n))
    if accepted is not None:
        _tensor(accepted, "accepted", _I32, (B,))
    # requests are decided at the same time: an output in place of an input
    # only where each request reads its own element alone
    inputs = {"draft_tokens": drafts, "uniforms": uniforms, "num_drafts": counts}
    same = tokens is not None and B == 1 and tokens.data_ptr() == drafts.data_ptr()
    _apart(tokens, "tokens", dict(inputs, accepted=accepted, draft_tokens=None if same else drafts))
    same = accepted is not None and counts is not None and accepted.data_ptr() == counts.data_ptr()
    _apart(accepted, "accepted", dict(inputs, num_drafts=None if same else counts))
    _place(target, drafts, uniforms, draft_probs, counts, tokens, accepted)


def _verify(name, target, drafts, uniforms, draft_probs, counts, tokens, accepted, stream):
    greedy = name == "msa_verify_greedy"
    try:
        (B, n, V), (t_req, t_row, one) = target.shape, target.stride()
        dev = target.get_device()
        sound = (
            one == 1 and n > 0 and target.dtype in _TYPES and drafts.shape == (B, n - 1)
            and drafts.dtype is torch.int32 and drafts.is_contiguous()
            and (greedy or (uniforms.shape == (B, n) and uniforms.dtype is torch.float32
                            and uniforms.is_contiguous() and uniforms.get_device() == dev))
            and (draft_probs is None
                 or (draft_probs.shape == (B, n - 1, V) and draft_probs.dtype is target.dtype
                     and draft_probs.stride(2) == 1 and draft_probs.get_device() == dev))
            and (counts is None or (counts.shape == (B,) and counts.dtype is torch.int32
                                    and counts.is_contiguous() and counts.get_device() == dev))
            and tokens is None and accepted is None and dev >= 0
            and dev == drafts.get_device() == torch._C._cuda_getDevice())
    except _NOT_SOUND:
        sound = False
    if not sound:
        _check_verify(greedy, target, drafts, uniforms, draft_probs, counts, tokens, accepted)
    handle = _handle(stream, dev)
    if tokens is None:
        tokens = _new((B, n), torch.int32, dev, handle)
    if accepted is None:
        accepted = _new((B,), torch.int32, dev, handle)
    if greedy:
        rc = load().msa_verify_greedy(target.data_ptr(), t_req, t_row, _TYPES[target.dtype],
                                      drafts.data_ptr(), _ptr(counts), B, n, V,
                                      tokens.data_ptr(), accepted.data_ptr(), handle)
    else:
        d_ptr, d_req, d_row = None, 0, 0
        if draft_probs is not None and n > 1:
            d_ptr = draft_probs.data_ptr()
            d_req, d_row, _ = draft_probs.stride()
        rc = load().msa_verify(target.data_ptr(), t_req, t_row, d_ptr, d_req, d_row,
                               _TYPES[target.dtype], drafts.data_ptr(), uniforms.data_ptr(),
                               _ptr(counts), B, n, V, tokens.data_ptr(), accepted.data_ptr(),
                               handle)
    if rc:
        _check(rc, name)
    return tokens, accepted


def msa_verify(target_probs, draft_tokens, uniforms, draft_probs=None, num_drafts=None,
               tokens=None, accepted=None, stream=None):
    """Which drafted tokens stand, and the token that follows them.
    target_probs [B, n, V] and draft_probs [B, n - 1, V] in fp32, bf16 or fp16
    (strided rows allowed; no draft_probs: the drafts were certain),
    draft_tokens int32 [B, n - 1], uniforms fp32 [B, n] in [0, 1), num_drafts
    int32 [B] or None for n - 1 each; accepted may be num_drafts itself, the
    outputs share no other memory with the inputs.  Returns (tokens int32
    [B, n]: the drafts that stand, the next token, -1; accepted int32 [B])."""
    return _verify("msa_verify", target_probs, draft_tokens, uniforms, draft_probs, num_drafts,
                   tokens, accepted, stream)


def msa_verify_greedy(target, draft_tokens, num_drafts=None, tokens=None, accepted=None,
                      stream=None):
    """msa_verify with a draft standing where it is the first of the largest
    values of its row of target [B, n, V] (logits or probabilities), and the
    best token following.  Returns (tokens, accepted)."""
    return _verify("msa_verify_greedy", target, draft_tokens, None, None, num_drafts, tokens,
                   accepted, stream)
