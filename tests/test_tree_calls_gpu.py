"""The two ways that a tree call takes to the library, the compiled module's and
the one with status, which checks its arguments one by one, give the same, and
refuse the same."""
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa

pytestmark = pytest.mark.gpu

i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
ORDER = {  # the calls and their arguments
    "rope": ("msa_rope_write", ("rope", "q", "k", "v", "kv", "q_scale", "k_scale", "v_scale", "block_table", "cu_seqlens_q", "cu_seqlens_k", "positions")),
    "rope4": ("msa_rope_write_nvfp4", ("rope", "q", "k", "v", "kv4", "q_scale", "k_scale", "v_scale", "block_table", "cu_seqlens_q", "cu_seqlens_k", "positions")),
    "mask": ("msa_tree_mask", ("parents", "cu_seqlens_q", "cu_seqlens_k", "max_seqlen_q")),
    "attend": ("msa_tree_attention", ("q", "kv", "q_scale", "k_scale", "v_scale", "softmax_scale", "block_table", "cu_seqlens_q", "cu_seqlens_k", "mask",
                                      "prefix_pages", "max_seqlen_q", "max_seqlen_k", "want_lse")),
    "accept": ("msa_tree_accept", ("draft_tokens", "parents", "chosen", "cu_seqlens_q", "cu_seqlens_k", "max_seqlen_q", "kv", "block_table")),
    "accept4": ("msa_tree_accept_nvfp4", ("draft_tokens", "parents", "chosen", "cu_seqlens_q", "cu_seqlens_k", "max_seqlen_q", "kv", "block_table")),
    "logprobs": ("msa_logprobs", ("logits", "tokens", "top")),
}


def _arguments(name):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    B, n, hq, hkv = 3, 9, 6, 2
    T = B * n
    cu_q, cu_k = i32([i * n for i in range(B + 1)]), i32([i * 200 for i in range(B + 1)])
    table = torch.randperm(B * 2, generator=g, device="cuda").to(torch.int32).view(B, 2)
    x = rand(T, hq + 2 * hkv, 128).bfloat16()
    kv = (rand(B * 2, hkv, 128, 256) / 0.013).to(torch.float8_e4m3fn)
    kv4 = torch.randint(0, 120, (B * 2, hkv, 2, 9216), generator=g, device="cuda", dtype=torch.uint8)
    parents = i32(([-1] + [i // 2 for i in range(n - 1)]) * B)
    drafts, chosen = (torch.randint(0, 2, (T,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2))
    mask = msa.msa_tree_mask(parents, cu_q, cu_k, n, status=i32([0]))[0]
    lens = {"cu_seqlens_q": cu_q, "cu_seqlens_k": cu_k}
    rotate = {"rope": msa.MsaRope([0.7 ** j for j in range(32)]), "q": x[:, :hq], "k": x[:, hq:hq + hkv], "v": x[:, hq + hkv:], "q_scale": 0.0131,
              "k_scale": 0.0127, "v_scale": 0.0149, "block_table": table, "positions": None, **lens}
    tree = {"draft_tokens": drafts, "parents": parents, "chosen": chosen, "max_seqlen_q": n, "block_table": table, **lens}
    return {
        "rope": lambda: {**rotate, "kv": kv.clone()},
        "rope4": lambda: {**rotate, "kv4": kv4.clone()},
        "mask": lambda: {"parents": parents, "max_seqlen_q": n, **lens},
        "attend": lambda: {"q": (x[:, :hq].float() / 0.013).to(torch.float8_e4m3fn), "kv": kv, "q_scale": 0.0131, "k_scale": 0.0127, "v_scale": 0.0149,
                           "softmax_scale": 0.09, "block_table": table, "mask": mask, "prefix_pages": 0, "max_seqlen_q": n, "max_seqlen_k": 200,
                           "want_lse": True, **lens},
        "accept": lambda: {**tree, "kv": [kv.clone(), kv.clone()]},
        "accept4": lambda: {**tree, "kv": [kv4.clone(), kv4.clone(), kv4.clone()]},
        "logprobs": lambda: {"logits": rand(T, 777), "tokens": drafts, "top": 4},
    }[name]()


def _call(name, args, **kw):
    f, order = ORDER[name]
    return getattr(msa, f)(**{k: args[k] for k in order}, **kw)


def _all(out, args):
    """The bytes of a call's outputs and of the pools that it wrote."""
    outs = list(out) if isinstance(out, tuple) else [out]
    pools = [args.get("kv"), args.get("kv4")]
    outs += [p for x in pools if x is not None for p in (x if isinstance(x, (list, tuple)) else [x])]
    return [None if t is None else (t.shape, t.dtype, t.contiguous().view(torch.uint8).cpu()) for t in outs]


def _same(a, b):
    return len(a) == len(b) and all((x is None) == (y is None) and (x is None or (x[:2] == y[:2] and torch.equal(x[2], y[2]))) for x, y in zip(a, b))


def _slow(name):  # logprobs has no status; a stream given by hand goes the same way
    return {"stream": torch.cuda.current_stream()} if name == "logprobs" else {"status": i32([0])}


FORMS = [(name, None, None) for name in ORDER] + [
    ("rope", "q_scale", None), ("rope4", "q_scale", None), ("rope", "q", None), ("rope", "positions", lambda a: torch.arange(27, device="cuda").int()),
    ("rope", "positions", lambda a: torch.arange(54, device="cuda").int().view(2, 27)), ("rope", "k", lambda a: a["k"].clone()),
    ("rope", "kv", lambda a: a["kv"].view(torch.uint8)), ("rope", "q", lambda a: a["q"][:, :0]),
    ("attend", "want_lse", lambda a: False), ("attend", "want_lse", lambda a: 1), ("attend", "want_lse", lambda a: 0),
    ("attend", "q", lambda a: a["q"].view(torch.uint8)), ("attend", "softmax_scale", lambda a: 1), ("attend", "max_seqlen_k", lambda a: 256),
    ("mask", "max_seqlen_q", lambda a: 200),
    ("accept", "kv", None), ("accept", "kv", lambda a: a["kv"][0]), ("accept", "kv", lambda a: tuple(a["kv"])), ("accept", "kv", lambda a: []),
    ("accept", "kv", lambda a: torch.stack([p.view(torch.uint8) for p in a["kv"]])), ("accept", "max_seqlen_q", lambda a: 256),
    ("logprobs", "tokens", None), ("logprobs", "top", lambda a: 0), ("logprobs", "top", lambda a: 32),
    ("logprobs", "logits", lambda a: a["logits"].half()), ("logprobs", "logits", lambda a: a["logits"][:, 3:700]),
    ("logprobs", "logits", lambda a: a["logits"][:1].expand(27, -1)), ("logprobs", "logits", lambda a: a["logits"][:, 5:6]),
]


@pytest.mark.parametrize("form", range(len(FORMS)))
def test_both_ways_give_the_same(form):
    name, key, change = FORMS[form]
    got = []
    for kw in ({}, _slow(name)):
        args = _arguments(name)
        if key:
            args[key] = change(args) if change else None
        if key == "q" and args["q"] is None:
            assert _call(name, args, **kw) is None
            got.append(_all((), args))
        else:
            got.append(_all(_call(name, args, **kw), args))
    assert _same(*got)


@pytest.mark.parametrize("name", ["mask", "accept", "logprobs"])
def test_outputs_of_one_allocation_lie_apart(name):
    outs = _call(name, _arguments(name))
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in outs)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])) and all(t.is_contiguous() and t.data_ptr() % 256 == 0 for t in outs)
    want = [t.clone() for t in outs]
    for i, t in enumerate(outs):
        t.add_(1)
        assert all(torch.equal(o, w) for o, w in zip(outs[i + 1:], want[i + 1:]))
    last, value = outs[-1], outs[-1].clone()
    del outs, t
    torch.cuda.synchronize()
    other = [torch.zeros(1 << 16, device="cuda") for _ in range(8)]  # noqa: F841
    assert torch.equal(last, value)


@pytest.mark.parametrize("name", ORDER)
def test_both_ways_refuse_the_same(name):
    """Every tensor of a call as another type, shape, order, place or nothing; every number out of range."""
    changes = [lambda t: t.double(), lambda t: t.cpu(), lambda t: t[:-1], lambda t: t[None], lambda t: t.transpose(0, -1) if t.dim() > 1 else t.repeat(2)[::2],
               lambda t: t.repeat_interleave(2, -1)[..., ::2], lambda t: t[..., :-1], lambda t: None, lambda t: "no", lambda t: t.to_sparse()]
    numbers = [-1, 257, 1 << 40, 1 << 70, 0, 0.0, -0.5, float("nan"), float("inf"), 2.5, True, None, "no"]

    def outcome(key, value, kw):
        args = _arguments(name)
        try:
            args[key] = value(args[key])
        except Exception:  # no such form of it
            return "none"
        try:
            out = _call(name, args, **kw)
        except Exception as e:
            return type(e).__name__
        torch.cuda.synchronize()
        return None if out is None else tuple(None if t is None else t.shape for t in (out if isinstance(out, tuple) else (out,)))

    wrong = []
    for key, was in _arguments(name).items():
        if isinstance(was, torch.Tensor):
            tries = changes
        elif isinstance(was, list):
            tries = [lambda t, c=c: [t[0], c(t[1])] for c in changes] + [lambda t: [t[0], t[0]], lambda t: t * 100, lambda t: [t[0], None], lambda t: "no"]
        elif was is None or isinstance(was, msa.MsaRope):
            tries = [lambda t: "no", lambda t: 3]
        else:
            tries = [lambda t, x=x: x for x in numbers]
        for i, change in enumerate(tries):
            a, b = outcome(key, change, {}), outcome(key, change, _slow(name))
            if isinstance(a, str) != isinstance(b, str) or (not isinstance(a, str) and a != b):
                wrong.append((key, i, a, b))
    assert not wrong, wrong
