"""Sampling several continuations of each prompt with drafted trees, as an engine makes the calls: prompts prefilled
into pages that the ledger gave, forked into samples, a token for each behind the shared pages, then rounds of trees:
rows grown, the nodes' keys written, attended to, verified, the accepted ones moved to their places and the rest
given back; at last everything freed.  A plain cache of dense tensors goes beside it; each step's attention is compared
with plain torch on the keys that the cache really holds, so that every tolerance is one step's own (bf16's half step
is 2^-8), and keys, lengths and tokens have to be equal."""
import math
import random

import pytest
import torch

from test_gpu_serving_step import D, H, HK, P, attend, near
from test_gpu_verify import reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
V = 50


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Engine:
    """The paged cache and its ledger, and beside them each row's keys and values as dense tensors."""

    def __init__(self, b2pa, rows, pages, width, seed):
        self.b2pa, self.R, self.N = b2pa, rows, pages
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.k, self.v = (torch.full((pages, HK, P, D), math.nan, dtype=BF, device=DEV) for _ in "kv")
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
        self.seq = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.keys = [torch.zeros((0, HK, D), dtype=BF, device=DEV) for _ in range(rows)]
        self.vals = list(self.keys)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device=DEV).to(BF)

    def write(self, rows, news):
        """Grow the rows by news[i] tokens and write their keys and values; returns (q, k, v) of all of them."""
        old = self.seq.tolist()
        self.b2pa.grow_pages(self.table, self.seq, self.refs, ints(rows), ints([old[r] + n for r, n in zip(rows, news)]), P)
        q, k, v = self.normal(sum(news), H, D), self.normal(sum(news), HK, D), self.normal(sum(news), HK, D)
        table = self.table.tolist()
        loc = [table[r][x // P] * P + x % P for r, n in zip(rows, news) for x in range(old[r], old[r] + n)]
        self.b2pa.append_kv(k, v, (self.k, self.v), ints(loc))
        return q, k, v

    def held(self, r, n):
        """The first n keys and values that row r's pages hold."""
        pg = self.table[r, : -(-n // P)].long()
        return tuple(x[pg].transpose(1, 2).reshape(-1, HK, D)[:n] for x in (self.k, self.v))

    def same(self, rows):
        lens = self.seq.tolist()
        for r in rows:
            assert lens[r] == self.keys[r].shape[0]
            k, v = self.held(r, lens[r])
            assert torch.equal(k, self.keys[r]) and torch.equal(v, self.vals[r])
        used = torch.zeros(self.N, dtype=torch.int32)
        for r in range(self.R):
            for pg in self.table[r, : -(-lens[r] // P)].tolist():
                used[pg] += 1
        assert torch.equal(used, self.refs.cpu())


@pytest.mark.parametrize("draft", [False, True])
def test_samples_with_drafted_trees(cuda_lib, draft):
    b2pa, r = cuda_lib, random.Random(7)
    e = Engine(b2pa, 12, 90, 20, 5)
    prompts = [70, 33]
    scale = 1 / math.sqrt(D)
    # the prompts
    q, k, v = e.write([0, 1], prompts)
    cum = ints([0, 70, 103])
    out = b2pa.context_attention(q, (e.k, e.v), e.table[:2], e.seq[:2], 70, 70, scale, 1.0, cum)
    for b, (lo, hi) in enumerate(((0, 70), (70, 103))):
        e.keys[b], e.vals[b] = k[lo:hi].clone(), v[lo:hi].clone()
        see = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device=DEV).tril()
        near(out[lo:hi], *attend(q[lo:hi], e.keys[b], e.vals[b], see), 2)
    e.same([0, 1])
    # their samples: four of the first, three of the second; the prompts go, their pages stay with the samples
    parents, samples = [0, 0, 0, 0, 1, 1, 1], [2, 3, 4, 5, 6, 7, 8]
    src, dst = b2pa.fork_pages(e.table, e.seq, e.refs, ints(parents), ints(samples), P)
    b2pa.copy_pages((e.k, e.v), src, dst)
    for a, b in zip(parents, samples):
        e.keys[b], e.vals[b] = e.keys[a], e.vals[a]
    e.same([0, 1] + samples)
    b2pa.free_pages(e.table, e.seq, e.refs, ints([0, 1]), P)
    e.keys[0] = e.keys[1] = e.vals[0] = e.vals[1] = e.keys[0][:0]
    e.same([0, 1] + samples)
    # a token each, behind the pages that are shared
    whole = [n // P for n in prompts]
    q, k, v = e.write(samples, [1] * 7)
    for i, s in enumerate(samples):
        e.keys[s], e.vals[s] = torch.cat([e.keys[s], k[i : i + 1]]), torch.cat([e.vals[s], v[i : i + 1]])
    e.same(samples)
    own = torch.stack([e.table[s, whole[p] : whole[p] + 12] for p, s in zip(parents, samples)])
    shared = torch.stack([e.table[2, :4], torch.cat([e.table[6, :2], ints([-1, -1])])])
    lens = ints([n + 1 - whole[p] * P for p in parents for n in [prompts[p]]])
    out = b2pa.prefix_attention(q, (e.k, e.v), shared, ints([w * P for w in whole]), ints([0, 4, 7]), own, lens, 1, 64, 16,
                                scale, 1.0, ints(range(8)), max_group_q_len=4)
    for i, s in enumerate(samples):
        see = torch.ones((1, e.keys[s].shape[0]), dtype=torch.bool, device=DEV)
        near(out[i : i + 1], *attend(q[i : i + 1], e.keys[s], e.vals[s], see), 2)
    # rounds of trees
    for turn in range(4):
        ns = [r.randint(1, 9) for _ in samples]
        ctx = e.seq.tolist()
        q, k, v = e.write(samples, ns)
        cums = [sum(ns[:i]) for i in range(len(ns) + 1)]
        up, masks = [], []
        for n in ns:
            m = torch.eye(n, dtype=torch.bool)
            for i in range(n):
                up.append(r.randint(max(0, i - 3), i - 1) if i else -1)
                if i:
                    m[i] |= m[up[-1]]
            masks.append(m)
        words = torch.cat([(m.long() << torch.arange(m.shape[0])).sum(1) for m in masks])[:, None].to(torch.int32).to(DEV)
        rows = e.table[samples[0] : samples[-1] + 1]
        seqs = e.seq[samples[0] : samples[-1] + 1].clone()
        out = b2pa.tree_attention(q, (e.k, e.v), rows, seqs, words, max(ns), int(seqs.max()), scale, 1.0, ints(cums))
        for i, s in enumerate(samples):
            lo, hi = cums[i], cums[i + 1]
            see = torch.cat([torch.ones((ns[i], ctx[s]), dtype=torch.bool), masks[i]], 1).to(DEV)
            near(out[lo:hi], *attend(q[lo:hi], torch.cat([e.keys[s], k[lo:hi]]), torch.cat([e.vals[s], v[lo:hi]]), see), 2)
        # what a model would make of it: the target's probabilities, tokens that the draft drew or chose
        z = torch.randn((cums[-1], V), generator=e.g, device=DEV) * 2
        p, qd = torch.softmax(z + 0.5 * torch.randn(z.shape, generator=e.g, device=DEV), -1), torch.softmax(z, -1)
        at = torch.tensor([max(u, 0) + cums[i] for i in range(len(ns)) for u in up[cums[i] : cums[i + 1]]], device=DEV)
        tokens = torch.multinomial(qd[at], 1, generator=e.g)[:, 0].int() if draft else qd[at].argmax(-1).int()
        u, last = torch.rand(cums[-1], generator=e.g, device=DEV), torch.rand(len(ns), generator=e.g, device=DEV)
        acc, cnt, nxt = b2pa.verify_trees(p, tokens, ints(up), u, last, max(ns), ints(cums), draft_probs=qd if draft else None)
        want = reference(p, qd if draft else None, tokens.tolist(), up, u.tolist(), last.tolist(), ns)
        lens = b2pa.compact_kv((e.k, e.v), rows, seqs, ints(cums), acc, cnt)
        b2pa.grow_pages(e.table, e.seq, e.refs, ints(samples), lens, P)
        for i, (s, (path, token)) in enumerate(zip(samples, want)):
            assert acc[i].tolist()[: len(path)] == path and int(nxt[i]) == token and int(cnt[i]) == len(path)
            pick = torch.tensor(path, device=DEV) + cums[i]
            e.keys[s], e.vals[s] = torch.cat([e.keys[s], k[pick]]), torch.cat([e.vals[s], v[pick]])
        e.same(samples)
        assert b2pa.device_status() == 0
    b2pa.free_pages(e.table, e.seq, e.refs, ints(samples), P)
    assert int(e.refs.sum()) == 0 and int(e.seq.sum()) == 0
    assert b2pa.device_status() == 0
