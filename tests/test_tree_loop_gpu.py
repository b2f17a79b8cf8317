"""Decoding with trees of drafted tokens, the calls together: prompts rotated
and written behind a shared document, then steps of (mask and positions, rotate
and write the tree, attend in each layer, log probabilities, accept and move the
path's rows), each on the state that the step before left.

Every step's attention is compared in 64 bits (tolerance: see
test_prefix_attention_gpu), the log probabilities and the walk with plain forms,
and in the end the caches with ones into which the same text is written at once.
Then the same steps run as a captured graph and give the same."""
import numpy as np
import pytest
import torch

import block_sparse_attention_prefill_gb300 as msa
from test_tree_gpu import _compare, _seen, _walk

pytestmark = pytest.mark.gpu

B, HQ, HKV, VOCAB, PREFIX, STEPS, LAYERS = 5, 8, 2, 97, 2, 6, 3
PROMPTS = (1, 120, 126, 200, 61)
QS, KS, VS, SM = 0.0131, 0.0127, 0.0149, 128 ** -0.5  # those of the tests whose comparison is used
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 4, 4, 5, 7]  # a fixed tree
N, DOC = len(PARENTS), PREFIX * 128
MAX_K = DOC + max(PROMPTS) + STEPS * N + N


class Server:
    def __init__(self):
        r = np.random.RandomState(0)
        g = torch.Generator(device="cuda")
        g.manual_seed(0)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        width = -(-MAX_K // 128)
        self.pages = PREFIX + B * (width - PREFIX) + 2
        perm = r.permutation(self.pages).astype(np.int32)
        table = np.empty((B, width), np.int32)
        table[:, :PREFIX] = perm[:PREFIX]
        table[:, PREFIX:] = perm[PREFIX:PREFIX + B * (width - PREFIX)].reshape(B, -1)
        self.table = torch.from_numpy(table).cuda()
        self.rope = msa.MsaRope([1e4 ** -(j / 32) for j in range(32)], q_norm=1 + 0.1 * rand(128), k_norm=1 + 0.1 * rand(128))
        self.pools = self.fresh()
        # a model by tables: what the projections of a token are in each layer, the logits of the last layer's output
        self.qkv = rand(LAYERS, VOCAB, HQ + 2 * HKV, 128).bfloat16()
        self.w = rand(VOCAB, HQ * 128) / 4
        self.guess = 2 * rand(VOCAB, VOCAB)
        self.text = torch.randint(VOCAB, (B, MAX_K), generator=g, device="cuda")
        self.text[:, :DOC] = self.text[0, :DOC]
        self.lens = torch.tensor([DOC + p for p in PROMPTS], dtype=torch.int32, device="cuda")
        self.last = torch.randint(VOCAB, (B,), generator=g, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cu_q = torch.arange(B + 1, dtype=torch.int32, device="cuda") * N
        self.parents = torch.tensor(PARENTS * B, dtype=torch.int32, device="cuda")

    def fresh(self):
        return [torch.full((self.pages, HKV, 128, 256), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(LAYERS)]  # NaN where nothing is written

    def put(self, layer, pool, tokens, cu_q, cu_k, table, positions=None):
        x = self.qkv[layer][tokens]
        return msa.msa_rope_write(self.rope, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], pool, QS, KS, VS, table, cu_q, cu_k, positions=positions,
                                  status=self.status)

    def prefill(self, pools, text, lens):
        cu = lambda v: torch.tensor(np.concatenate([[0], np.cumsum(v)]), dtype=torch.int32, device="cuda")  # noqa: E731
        for i, pool in enumerate(pools):
            self.put(i, pool, text[0, :DOC], cu([DOC]), cu([DOC]), self.table[:1])
            rest = torch.cat([text[b, DOC:n] for b, n in enumerate(lens)])
            self.put(i, pool, rest, cu([n - DOC for n in lens]), cu(lens), self.table)

    def step(self):
        """One step, in tensors alone; updates lens and last in place."""
        cu_k = torch.nn.functional.pad(torch.cumsum(self.lens + N, 0, dtype=torch.int32), (1, 0))
        mask, positions = msa.msa_tree_mask(self.parents, self.cu_q, cu_k, N, status=self.status)
        # the draft model: a node's children are its likeliest followers, but for a shift by the length
        x = [self.last]
        for i in range(1, N):
            nth = PARENTS[:i].count(PARENTS[i])
            x.append((self.guess[x[PARENTS[i]]].topk(3).indices[:, nth] + (self.lens % 4 == 0)) % VOCAB)
        drafts = torch.stack(x, 1).reshape(-1)
        qs, outs = [], []
        for i, pool in enumerate(self.pools):
            q = self.put(i, pool, drafts, self.cu_q, cu_k, self.table, positions)
            out, lse = msa.msa_tree_attention(q, pool, QS, KS, VS, SM, self.table, self.cu_q, cu_k, mask, PREFIX, N, MAX_K, status=self.status)
            qs.append(q), outs.append((out, lse))
        logits = torch.matmul(outs[-1][0].reshape(B * N, -1).float(), self.w.T) + self.guess[drafts]
        logprobs, ranks, entropy, best, values = msa.msa_logprobs(logits, drafts.int(), top=3)
        chosen = best[:, 0].contiguous()
        before = [p.clone() for p in self.pools]
        tokens, accepted, path = msa.msa_tree_accept(drafts.int(), self.parents, chosen, self.cu_q, cu_k, N, kv=self.pools, block_table=self.table,
                                                     status=self.status)
        old = self.lens.clone()
        self.lens += accepted + 1
        last = self.last.clone()
        self.last.copy_(tokens.gather(1, accepted.long()[:, None])[:, 0])
        return {"mask": mask, "positions": positions, "drafts": drafts, "qs": qs, "outs": outs, "logits": logits, "logprobs": logprobs, "ranks": ranks,
                "entropy": entropy, "best": best, "chosen": chosen, "before": before, "tokens": tokens, "accepted": accepted, "path": path, "old": old,
                "last": last}


def test_steps_match_plain_forms_and_a_graph():
    s = Server()
    s.prefill(s.pools, s.text, s.lens.tolist())
    start = [t.clone() for t in (*s.pools, s.lens, s.last)]
    text = s.text.clone()  # what was said
    history, stood = [], 0
    for _ in range(STEPS):
        r = s.step()
        assert s.status.item() == 0
        old = r["old"].tolist()
        depth = [int(d) - 1 for d in _seen(PARENTS).sum(1)]
        assert r["positions"].tolist() == [n + d for n in old for d in depth]
        for i in range(LAYERS):
            w = {"q": r["qs"][i], "kv": r["before"][i].view(torch.float8_e4m3fn), "table": s.table, "q_lens": [N] * B, "seqs": [n + N for n in old]}
            _compare(w, [_seen(PARENTS)] * B, r["outs"][i])
        x = r["logits"].double()
        z = torch.log_softmax(x, -1)
        assert ((r["logprobs"] - z.gather(1, r["drafts"][:, None])[:, 0]).abs() < 1e-5).all()
        assert ((r["entropy"] + (z.exp() * z).sum(-1)).abs() < 1e-5).all()
        assert torch.equal(r["best"].long(), torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :3])
        drafts, chosen = r["drafts"].view(B, N).tolist(), r["chosen"].view(B, N).tolist()
        for b in range(B):
            path = _walk(PARENTS, drafts[b], chosen[b])
            assert r["path"][b].tolist() == path + [-1] * (N - len(path)) and r["accepted"][b] == len(path) - 1
            said = [drafts[b][i] for i in path]
            assert said[0] == r["last"][b] and r["tokens"][b, :len(path)].tolist() == said[1:] + [chosen[b][path[-1]]]
            text[b, old[b]:old[b] + len(said)] = torch.tensor(said, device="cuda")
            stood += len(path) - 1
        history.append([r[k].clone() for k in ("tokens", "accepted", "path")])
    assert 0 < stood < STEPS * B * 4  # drafts stood and fell
    # the caches hold what the same text written at once gives
    fresh = s.fresh()
    lens = s.lens.tolist()
    s.prefill(fresh, text, lens)
    for pool, want in zip(s.pools, fresh):
        for b, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            page = s.table[b].long()[pos // 128]
            assert torch.equal(pool[page, :, pos % 128], want[page, :, pos % 128])
    end = [p.clone() for p in s.pools]
    # the same as a captured graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = s.step()
    for t, v in zip((*s.pools, s.lens, s.last), start):
        t.copy_(v)
    for want in history:
        graph.replay()
        assert all(torch.equal(r[k], v) for k, v in zip(("tokens", "accepted", "path"), want))
    assert all(torch.equal(p, v) for p, v in zip(s.pools, end)) and s.status.item() == 0
