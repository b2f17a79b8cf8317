"""Speculative decoding with the serving calls together: prompts written into
the paged cache behind a shared document, then steps of (write the new tokens'
K and V, attend, verify the drafts), each on the state that the step before
left; positions of drafts that fell are written over by the next step.

Every step's operators are compared with plain forms on the inputs they had:
the whole pool equal, the attention in 64 bits (tolerance: see
test_prefix_attention_gpu), the tokens equal.  Then the same steps run as a
captured graph and give the same."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_prefix_attention_gpu import _compare
from test_verify_gpu import _reference as verify_reference

pytestmark = pytest.mark.gpu

B, DRAFTS, HQ, HKV, VOCAB, PREFIX, STEPS = 5, 3, 8, 2, 40, 3, 6
PROMPTS = (1, 127, 128, 200, 61)
QS, KS, VS, SM = 0.0131, 0.0127, 0.0149, 128 ** -0.5  # those of the tests whose comparison is used
N, DOC = DRAFTS + 1, PREFIX * 128
MAX_K = DOC + max(PROMPTS) + STEPS * N


class Server:
    def __init__(self):
        r = np.random.RandomState(0)
        g = torch.Generator(device="cuda")
        g.manual_seed(0)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        width = -(-MAX_K // 128)
        pages = PREFIX + B * (width - PREFIX) + 2
        perm = r.permutation(pages).astype(np.int32)
        table = np.empty((B, width), np.int32)
        table[:, :PREFIX] = perm[:PREFIX]
        table[:, PREFIX:] = perm[PREFIX:PREFIX + B * (width - PREFIX)].reshape(B, -1)
        self.table = torch.from_numpy(table).cuda()
        self.pool = torch.full((pages, HKV, 128, 256), 0x7F, dtype=torch.uint8, device="cuda")  # NaN where nothing is written
        # a model by tables: K, V, Q of a token, the logits of an output, the draft model's logits
        self.k_of, self.v_of = rand(VOCAB, HKV, 128).bfloat16(), rand(VOCAB, HKV, 128).bfloat16()
        self.q_of = (rand(VOCAB, HQ, 128) / QS).to(torch.float8_e4m3fn)
        self.w = rand(VOCAB, HQ * 128) / 8
        self.draft_logits = 2 * rand(VOCAB, VOCAB)
        self.uniforms = torch.rand((STEPS, B, N), generator=g, device="cuda")
        # prompts
        self.text = torch.randint(VOCAB, (B, MAX_K), generator=g, device="cuda")
        self.text[:, :DOC] = self.text[0, :DOC]
        self.lens = torch.tensor([DOC + p for p in PROMPTS], dtype=torch.int32, device="cuda")
        self.last = torch.randint(VOCAB, (B,), generator=g, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cu_q = torch.arange(B + 1, dtype=torch.int32, device="cuda") * N
        self.ws = torch.empty(msa.prefix_attention_workspace_bytes(B, B * N, HQ, HKV, PREFIX, N, MAX_K), dtype=torch.uint8, device="cuda")

    def prefill(self):
        cu = lambda v: torch.tensor(np.concatenate([[0], np.cumsum(v)]), dtype=torch.int32, device="cuda")  # noqa: E731
        # the document once, for the first request; then all prompts, ragged, in one call
        doc = self.text[0, :DOC]
        msa.msa_kv_write(self.k_of[doc], self.v_of[doc], self.pool, KS, VS, self.table[:1], cu([DOC]), cu([DOC]), status=self.status)
        rest = torch.cat([self.text[b, DOC:DOC + p] for b, p in enumerate(PROMPTS)])
        msa.msa_kv_write(self.k_of[rest], self.v_of[rest], self.pool, KS, VS, self.table, cu(PROMPTS), cu([DOC + p for p in PROMPTS]), status=self.status)

    def step(self, uniforms):
        """One step, in tensors alone; updates lens and last in place."""
        x = [self.last]
        for _ in range(DRAFTS):  # the draft model's likeliest token but for a shift by the length
            x.append((self.draft_logits[x[-1]].argmax(-1) + (self.lens % 3 == 0)) % VOCAB)
        x = torch.stack(x, 1)
        cu_k = torch.nn.functional.pad(torch.cumsum(self.lens + N, 0, dtype=torch.int32), (1, 0))
        flat = x.reshape(-1)
        msa.msa_kv_write(self.k_of[flat], self.v_of[flat], self.pool, KS, VS, self.table, self.cu_q, cu_k, status=self.status)
        q = self.q_of.view(torch.uint8)[flat].view(torch.float8_e4m3fn)
        out, lse = msa.msa_prefix_attention(q, self.pool, QS, KS, VS, SM, self.table, self.cu_q, cu_k, PREFIX, N, MAX_K, workspace=self.ws,
                                            status=self.status)
        logits = (out.reshape(B * N, 1, -1).float() * self.w).sum(-1)
        probs = torch.softmax(logits + self.draft_logits[flat], -1).reshape(B, N, VOCAB)
        drafts = x[:, 1:].int().contiguous()
        draft_probs = torch.softmax(self.draft_logits[x[:, :-1]], -1)
        tokens, accepted = msa.msa_verify(probs, drafts, uniforms, draft_probs=draft_probs)
        self.lens += accepted + 1
        self.last.copy_(tokens.gather(1, accepted.long()[:, None])[:, 0])
        return {"x": x, "q": q, "out": out, "lse": lse, "probs": probs, "drafts": drafts, "draft_probs": draft_probs, "tokens": tokens,
                "accepted": accepted}


def _e4m3(x, scale):
    # (by a tensor: by a number torch multiplies with its reciprocal)
    return (x.float() / torch.tensor(scale, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def test_steps_match_plain_forms_and_a_graph():
    s = Server()
    s.prefill()
    start = (s.pool.clone(), s.lens.clone(), s.last.clone())
    pool = torch.full_like(s.pool, 0x7F)  # what the cache should hold

    def put(b, first, tokens):
        pos = torch.arange(first, first + len(tokens), device="cuda")
        page = s.table[b].long()[pos // 128]
        pool[page, :, pos % 128, :128] = _e4m3(s.k_of[tokens], KS)
        pool[page, :, pos % 128, 128:] = _e4m3(s.v_of[tokens], VS)

    for b, p in enumerate(PROMPTS):
        put(b, 0, s.text[b, :DOC + p])
    assert torch.equal(s.pool, pool)
    history, stood = [], 0
    for i in range(STEPS):
        lens = s.lens.tolist()
        r = s.step(s.uniforms[i])
        for b in range(B):
            put(b, lens[b], r["x"][b])
        assert torch.equal(s.pool, pool) and s.status.item() == 0
        _compare({"q": r["q"], "kv": s.pool.view(torch.float8_e4m3fn), "table": s.table, "q_lens": [N] * B, "seqs": [n + N for n in lens]},
                 (r["out"], r["lse"]))
        np32 = lambda t: t.cpu().numpy()  # noqa: E731
        tokens, accepted = verify_reference(np32(r["probs"]), np32(r["draft_probs"]), np32(r["drafts"]), np32(s.uniforms[i]), None)
        assert np.array_equal(np32(r["tokens"]), tokens) and np.array_equal(np32(r["accepted"]), accepted)
        history.append((r["tokens"].clone(), r["accepted"].clone()))
        stood += int(accepted.sum())
    assert 0 < stood < STEPS * B * DRAFTS  # both outcomes were met
    # the document reads back
    k, v = msa.msa_kv_read(s.pool, KS, VS, s.table, torch.tensor([0] + [DOC] * B, dtype=torch.int32, device="cuda"), DOC, dtype=torch.float32)
    code = _e4m3(s.k_of[s.text[0, :DOC]], KS).view(torch.float8_e4m3fn)
    assert torch.equal(k, code.float() * torch.tensor(KS, dtype=torch.float32, device="cuda"))

    # the same as a captured graph
    end = s.pool.clone()
    u = torch.empty_like(s.uniforms[0])
    u.copy_(s.uniforms[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = s.step(u)
    for t, v in zip((s.pool, s.lens, s.last), start):
        t.copy_(v)
    for i in range(STEPS):
        u.copy_(s.uniforms[i])
        graph.replay()
        assert torch.equal(r["tokens"], history[i][0]) and torch.equal(r["accepted"], history[i][1])
    assert torch.equal(s.pool, end) and s.status.item() == 0
