"""Attention of drafted token trees over a paged cache (b2pa_tree_attention) on
the GPU, against the formula in fp64.

Tolerance, with A = sum p|v| / sum p over the keys a row sees:
  the result's rounding to bf16: 2^-8 |o| (half a step);
  each probability's rounding to bf16, or to two e4m3 terms: 2^-8 A; the terms
  (an e4m3 step is 2^-9 at its smallest, half of it 2^-10, with the row's largest
  probability at 2^4 or more) stop at 2^-14 of it: 2^-14 p_max sum|v| / sum p;
  scores in fp32 (unit 2^-24, D + 8 roundings of products and sums): ds = 2^-24
  (D + 8) bmm1 max_j sum_d |q_d k_jd|, with e4m3 terms of q 2^-17 max|q| bmm1
  max_j sum_d |k_jd| more; a score's error changes its weight by that factor, in
  numerator and denominator: 2 ds A;
  the exponent's own rounding and approximation (|x| < 128, 2^-22): 2^-15 A."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


class Batch:
    """Trees ns over contexts: kvs keys each, the last of them the nodes'."""

    def __init__(self, ns, kvs, H, Hkv, D, P, layout="HND", cache="bf16", window=-1, sinks=False, seed=0, q_scale=1.0,
                 words=None, deep=False):
        g = torch.Generator().manual_seed(seed)
        self.ns, self.kvs, self.H, self.Hkv, self.D, self.P = ns, kvs, H, Hkv, D, P
        self.layout, self.window, self.cache = layout, window, cache
        used = [-(-k // P) for k in kvs]
        N = sum(used) + 3
        shape = (N, Hkv, P, D) if layout == "HND" else (N, P, Hkv, D)
        self.k, self.v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        if cache == "e4m3":
            self.k, self.v = (self.k * 50).to(F8), (self.v * 50).to(F8)
            self.bmm1, self.bmm2 = 1 / math.sqrt(D) / 50, 1 / 50
        else:
            self.k, self.v = self.k.to(BF), self.v.to(BF)
            self.bmm1, self.bmm2 = 1 / math.sqrt(D), 1.0
        self.pages = torch.randperm(N, generator=g).to(torch.int32)
        self.table = torch.full((len(ns), max(used + [1]) + 2), -7, dtype=torch.int32)  # padding is no page
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = self.pages[at : at + u]
            at += u
        self.seq = torch.tensor(kvs, dtype=torch.int32)
        self.cum = torch.tensor([sum(ns[:i]) for i in range(len(ns) + 1)], dtype=torch.int32)
        T = sum(ns)
        self.q = (torch.randn((T, H, D), generator=g) * q_scale).to(BF)
        self.sinks = torch.randn(H, generator=g) if sinks else None
        self.max_q, self.max_kv = max(ns + [0]), max(kvs + [0])
        W = words or max(1, -(-self.max_q // 32))
        r = random.Random(seed)
        self.sees = []  # per request [n, n]
        self.pos = torch.zeros(T, dtype=torch.int32)
        mask = torch.randint(-2 ** 31, 2 ** 31, (T, W), generator=g)  # bits from n on are ignored
        row = 0
        for n, kv in zip(ns, kvs):
            m = torch.zeros((n, n), dtype=torch.bool)
            for i in range(n):
                up = i - 1 if deep else r.randint(-1, i - 1)
                if up >= 0:
                    m[i] = m[up]
                m[i, i] = True
                self.pos[row + i] = kv - n + int(m[i].sum()) - 1
            self.sees.append(m)
            row += n
        self.mask = mask
        self.pack()

    def pack(self):
        row = 0
        for m in self.sees:
            n = m.shape[0]
            for i in range(n):
                for j in range(n):
                    w, s = j // 32, j % 32
                    v = int(self.mask[row + i, w]) & 0xFFFFFFFF
                    v = v | (1 << s) if m[i, j] else v & ~(1 << s)
                    self.mask[row + i, w] = v - (1 << 32) if v >= 1 << 31 else v
            row += n

    def view(self, b):
        """[n, kv] bool: the keys each node of request b sees."""
        n, kv = self.ns[b], self.kvs[b]
        row = int(self.cum[b])
        see = torch.zeros((n, kv), dtype=torch.bool)
        for i in range(n):
            pos = min(max(int(self.pos[row + i]), kv - n), kv - 1)
            lo = 0 if self.window < 0 else max(0, pos - self.window)
            see[i, lo : kv - n] = True
        see[:, kv - n :] = self.sees[b]
        return see

    def dev(self):
        d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        return dict(query=d(self.q), kv_cache=(d(self.k), d(self.v)), block_tables=d(self.table), seq_lens=d(self.seq),
                    tree_mask=d(self.mask.to(torch.int32)), max_q_len=self.max_q, max_kv_len=self.max_kv,
                    bmm1_scale=self.bmm1, bmm2_scale=self.bmm2, cum_seq_lens_q=d(self.cum),
                    positions=d(self.pos) if self.window >= 0 else None, window_left=self.window,
                    kv_layout=self.layout, sinks=d(self.sinks))

    def rows(self, pool, b):
        """[Hkv, kv, D] in fp64 of request b."""
        P = self.P
        pg = self.table[b, : -(-self.kvs[b] // P)].long()
        x = pool.view(torch.uint8)[pg].view(F8) if pool.dtype == F8 else pool[pg]
        x = x.to(DEV).to(torch.float64)
        x = x.transpose(1, 2) if self.layout == "HND" else x
        return x.reshape(-1, self.Hkv, self.D)[: self.kvs[b]].transpose(0, 1)

    def check(self, out):
        """Every row of `out` against the formula; keys a row does not see are left out, whatever they hold."""
        D, G = self.D, self.H // self.Hkv
        for b, n in enumerate(self.ns):
            if n == 0:
                continue
            k, v = self.rows(self.k, b), self.rows(self.v, b)
            see = self.view(b).to(DEV)
            q = self.q[int(self.cum[b]) : int(self.cum[b]) + n].to(DEV).double().transpose(0, 1)
            q = q.reshape(self.Hkv, G * n, D)
            see_r = see.repeat(G, 1)
            s = torch.where(see_r, torch.nan_to_num(q) @ torch.nan_to_num(k, posinf=0, neginf=0).transpose(1, 2) * self.bmm1,
                            -math.inf)
            top = s.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, 0.0, top)
            p = torch.exp(s - top)
            den = p.sum(-1, keepdim=True)
            if self.sinks is not None:
                sk = self.sinks.double().to(DEV).view(self.Hkv, G, 1).repeat_interleave(n, 2).view(self.Hkv, G * n, 1)
                den = torch.where(see_r.any(-1, keepdim=True), den + torch.exp(sk - top), den)
            fin = torch.isfinite(v)
            v0 = torch.where(fin, v, 0.0)
            o = p @ v0
            # what is not finite reaches the rows that see it
            if not fin.all():
                w = p > 0
                for kind in (torch.isnan(v), v == math.inf, v == -math.inf):
                    hit = (w.double() @ kind.double()) > 0
                    bad = math.nan if kind is not None and torch.isnan(v)[kind].any() else None
                    o = torch.where(hit, o + (math.nan if bad is not None else v[kind][0] if kind.any() else 0.0), o)
            live = den > 0
            den = torch.where(live, den, 1.0)
            o = o / den * self.bmm2
            A = (p @ v0.abs()) / den * self.bmm2
            smax = (torch.nan_to_num(q).abs() @ torch.nan_to_num(k, posinf=0, neginf=0).abs().transpose(1, 2)).masked_fill(
                ~see_r, 0).amax(-1, keepdim=True) * self.bmm1
            ds = 2.0 ** -24 * (D + 8) * smax
            extra = 0.0
            if self.cache == "e4m3":
                kmax = torch.nan_to_num(k).abs().sum(-1).amax(-1)[:, None, None]
                ds = ds + 2.0 ** -17 * torch.nan_to_num(q).abs().amax(-1, keepdim=True) * kmax * self.bmm1
                extra = 2.0 ** -14 * (see_r.double() @ v0.abs()) / den * self.bmm2
            tol = 2.0 ** -8 * o.abs() + A * (2.0 ** -8 + 2 * ds + 2.0 ** -15) + extra + 1e-30
            got = out[int(self.cum[b]) : int(self.cum[b]) + n].double().transpose(0, 1).reshape(self.Hkv, G * n, D)
            same = torch.where(torch.isfinite(o), (got - o).abs() <= tol,
                               torch.where(torch.isnan(o), torch.isnan(got), got == o))
            assert same.all(), (b, int((~same).sum()), float(torch.nan_to_num((got - o).abs() - tol, nan=9e9).max()))


CASES = {
    "one_node": dict(ns=[1], kvs=[1], H=1, Hkv=1, D=128, P=8),
    "chain_of_8": dict(ns=[8], kvs=[300], H=8, Hkv=2, D=128, P=32, deep=True),
    "no_context": dict(ns=[16, 5], kvs=[16, 5], H=8, Hkv=2, D=128, P=16),
    "ragged": dict(ns=[7, 0, 16, 1, 12], kvs=[700, 33, 1025, 128, 12], H=32, Hkv=8, D=128, P=32),
    "nhd_p64": dict(ns=[31, 32, 9], kvs=[500, 64, 2049], H=16, Hkv=4, D=128, P=64, layout="NHD"),
    "two_tiles": dict(ns=[64, 33, 3], kvs=[900, 400, 130], H=16, Hkv=2, D=128, P=128, seed=3),
    "several_items": dict(ns=[300, 65, 0, 1], kvs=[1500, 65, 10, 900], H=8, Hkv=1, D=128, P=16),
    "page_256": dict(ns=[10, 20], kvs=[1000, 257], H=4, Hkv=1, D=128, P=256),
    "heads_3": dict(ns=[20, 41], kvs=[333, 555], H=6, Hkv=2, D=128, P=32),
    "heads_5_d64": dict(ns=[24, 25, 13], kvs=[333, 100, 640], H=5, Hkv=1, D=64, P=16),
    "heads_16": dict(ns=[8, 9], kvs=[1333, 200], H=16, Hkv=1, D=64, P=32),
    "heads_32": dict(ns=[4, 3], kvs=[333, 200], H=32, Hkv=1, D=128, P=32),
    "heads_40": dict(ns=[4, 3, 9], kvs=[333, 200, 9], H=40, Hkv=1, D=128, P=32),
    "heads_128": dict(ns=[2, 3], kvs=[333, 200], H=128, Hkv=1, D=128, P=32),
    "heads_1_d64": dict(ns=[129, 70], kvs=[1333, 70], H=4, Hkv=4, D=64, P=8),
    "sinks": dict(ns=[16, 5], kvs=[800, 5], H=8, Hkv=2, D=128, P=32, sinks=True),
    "window": dict(ns=[16, 30, 4], kvs=[800, 95, 2000], H=8, Hkv=2, D=128, P=16, window=100),
    "window_0": dict(ns=[9], kvs=[900], H=8, Hkv=2, D=64, P=16, window=0, sinks=True),
    "window_sinks_d64": dict(ns=[32, 24], kvs=[1200, 700], H=64, Hkv=8, D=64, P=16, window=127, sinks=True),
    "window_long": dict(ns=[70, 2], kvs=[3000, 1500], H=8, Hkv=2, D=128, P=32, window=1000),
    "e4m3": dict(ns=[8, 3, 0, 5], kvs=[700, 300, 40, 1025], H=32, Hkv=8, D=128, P=32, cache="e4m3"),
    "e4m3_two_tiles": dict(ns=[64, 40], kvs=[900, 41], H=16, Hkv=4, D=128, P=64, layout="NHD", cache="e4m3", sinks=True),
    "e4m3_window": dict(ns=[20, 6], kvs=[600, 1500], H=10, Hkv=2, D=128, P=16, cache="e4m3", window=300),
    "e4m3_large_q": dict(ns=[20, 6], kvs=[600, 1500], H=8, Hkv=2, D=128, P=16, cache="e4m3", q_scale=3e4),
    "sharp": dict(ns=[20, 6], kvs=[600, 1500], H=8, Hkv=2, D=128, P=16, q_scale=8.0),
    "wide_mask": dict(ns=[20, 6], kvs=[600, 150], H=8, Hkv=2, D=128, P=16, words=5),
    # CUDA cores
    "generic_d16": dict(ns=[5, 0, 40], kvs=[9, 4, 300], H=4, Hkv=2, D=16, P=4, sinks=True),
    "generic_d80_p3": dict(ns=[5, 7], kvs=[90, 7], H=6, Hkv=2, D=80, P=3, layout="NHD", window=20),
    "generic_window_below_depth": dict(ns=[40, 7], kvs=[90, 30], H=4, Hkv=2, D=48, P=8, window=2, deep=True),
    "window_below_depth": dict(ns=[40, 7], kvs=[290, 30], H=4, Hkv=2, D=128, P=8, window=2, deep=True),
    "generic_d256": dict(ns=[33], kvs=[200], H=2, Hkv=1, D=256, P=16),
    "generic_e4m3_d64": dict(ns=[9, 2], kvs=[200, 77], H=4, Hkv=1, D=64, P=16, cache="e4m3"),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(cuda_lib, name):
    t = Batch(**CASES[name])
    out = cuda_lib.tree_attention(**t.dev())
    assert cuda_lib.device_status() == 0
    t.check(out)


@pytest.mark.parametrize("G,n", [(1, 1), (1, 64), (1, 65), (1, 128), (1, 129), (3, 20), (3, 21), (3, 41), (4, 1), (4, 2), (4, 16),
                                 (4, 17), (5, 12), (5, 13), (31, 2), (31, 3), (32, 1), (32, 2), (32, 3), (32, 5), (33, 1),
                                 (33, 4), (64, 2), (100, 1)])
def test_e4m3_tiles_at_their_edges(cuda_lib, G, n):
    """Row counts around those at which a tile holds its rows twice, once, and in two tiles."""
    t = Batch([n, max(1, n - 1), 1], [1500, 130, 700], 2 * G, 2, 128, 16, cache="e4m3", sinks=G % 2 == 0, seed=G + n)
    t.check(cuda_lib.tree_attention(**t.dev()))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("name", ["ragged", "window", "two_tiles", "e4m3"])
def test_generic_path_and_padding_rows(cuda_lib, name):
    """The CUDA-core path on tensor-core shapes; rows behind the last request stay as they were."""
    t = Batch(**CASES[name])
    d = t.dev()
    T = t.q.shape[0]
    d["query"] = torch.cat([d["query"], d["query"][:3]])
    d["tree_mask"] = torch.cat([d["tree_mask"], d["tree_mask"][:3]])
    if d["positions"] is not None:
        d["positions"] = torch.cat([d["positions"], d["positions"][:3]])
    for path in ("auto", "generic"):
        out = torch.full_like(d["query"], 5.0)
        cuda_lib.set_kernel_path(path)
        try:
            cuda_lib.tree_attention(**d, out=out)
        finally:
            cuda_lib.set_kernel_path("auto")
        t.check(out)
        assert (out[T:] == 5).all()


@pytest.mark.parametrize("cache,kv", [("bf16", 70000), ("e4m3", 70000), ("bf16", 19457)])
def test_long_context_cut_over_all_sms(cuda_lib, cache, kv):
    t = Batch([13], [kv], 8, 2, 128, 64, cache=cache, seed=5)
    d = t.dev()
    out = cuda_lib.tree_attention(**d)
    t.check(out)
    for _ in range(3):
        assert torch.equal(out, cuda_lib.tree_attention(**d))  # the same bits every time
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("kvs", [[512] * 24, [513] * 24, [1024] * 8, [1025] * 16, [640] * 33, [300] * 60, [4] * 40,
                                 [100, 500, 1000, 1100, 9000, 4] * 3, [100, 500, 1000, 1100, 9000, 4] * 9],
                         ids=lambda k: f"{len(k)}x{k[0]}")
def test_units_whole_and_cut(cuda_lib, cache, kvs):
    """Requests around the sizes up to which no CTA's share ends inside one, alone and among others."""
    t = Batch([4] * len(kvs), kvs, 16, 4, 128, 32, cache=cache, seed=len(kvs) + kvs[0])
    out = cuda_lib.tree_attention(**t.dev())
    assert cuda_lib.device_status() == 0
    t.check(out)
    assert torch.equal(out, cuda_lib.tree_attention(**t.dev()))


def test_many_requests(cuda_lib):
    r = random.Random(1)
    ns = [r.choice([0, 1, 2, 3, 5, 8]) for _ in range(900)]
    kvs = [max(n, r.randint(1, 300)) for n in ns]
    t = Batch(ns, kvs, 4, 2, 64, 16, seed=6)
    t.check(cuda_lib.tree_attention(**t.dev()))
    assert cuda_lib.device_status() == 0


def test_a_chain_is_the_decode_batch(cuda_lib):
    n, B = 4, 6
    t = Batch([n] * B, [50, 4, 700, 128, 129, 2000], 16, 4, 128, 32, deep=True, seed=8)
    d = t.dev()
    got = cuda_lib.tree_attention(**d)
    ref = cuda_lib.batch_decode(d["query"], d["kv_cache"], d["block_tables"].clamp(min=0), d["seq_lens"], t.max_kv,
                                t.bmm1, t.bmm2, q_len_per_req=n)
    t.check(got)
    t.check(ref)  # both within the same bounds of the formula


@pytest.mark.parametrize("cfg", [dict(H=8, Hkv=2, D=128, P=16), dict(H=32, Hkv=8, D=64, P=8, window=50),
                                 dict(H=16, Hkv=2, D=128, P=32, cache="e4m3"), dict(H=2, Hkv=1, D=48, P=8, window=50),
                                 dict(H=4, Hkv=2, D=128, P=32, cache="e4m3", window=50)],
                         ids=["bf16", "d64_window", "e4m3", "generic", "e4m3_rows_twice"])
@pytest.mark.parametrize("sinks", [False, True])
def test_rows_that_see_nothing(cuda_lib, cfg, sinks):
    t = Batch([12, 20], [12, 400], sinks=sinks, **cfg)
    t.sees[0][3] = False
    t.sees[0][0] = False  # no context either: nothing
    t.sees[1][7] = False  # the context alone
    t.pack()
    out = cuda_lib.tree_attention(**t.dev())
    assert (out[0] == 0).all() and (out[3] == 0).all()
    t.check(out)


@pytest.mark.parametrize("cfg", [dict(H=8, Hkv=2, D=128, P=16), dict(H=8, Hkv=2, D=64, P=16, window=40),
                                 dict(H=8, Hkv=2, D=128, P=16, cache="e4m3"), dict(H=16, Hkv=1, D=128, P=128),
                                 dict(H=4, Hkv=2, D=48, P=8, window=40), dict(H=4, Hkv=2, D=128, P=16, cache="e4m3"),
                                 dict(H=4, Hkv=2, D=128, P=16, cache="e4m3", window=40),
                                 dict(H=16, Hkv=1, D=128, P=128, cache="e4m3"), dict(H=8, Hkv=2, D=64, P=16, window=2, deep=True),
                                 dict(H=4, Hkv=2, D=48, P=8, window=2, deep=True)],
                         ids=["bf16", "d64_window", "e4m3", "two_tiles", "generic", "e4m3_rows_twice",
                              "e4m3_rows_twice_window", "e4m3_two_tiles", "d64_window_below_depth",
                              "generic_window_below_depth"])
@pytest.mark.parametrize("kv", [40, 260])
def test_what_unseen_keys_hold_does_not_matter(cuda_lib, cfg, kv):
    """NaN and infinities in V (and NaN in K) of sibling nodes, of page tails, of pages nobody uses and before a window."""
    n = 20
    t = Batch([n], [kv], seed=4, **cfg)
    # node 2 is seen by itself and by node 9 alone, node 5 by nobody
    m = t.sees[0]
    m[:, 2] = False
    m[2, 2] = m[9, 2] = True
    m[:, 5] = False
    t.pack()
    P, bad = t.P, t.v
    hnd = t.layout == "HND"

    def put(pool, key, d, x):
        pg, slot = int(t.table[0, key // P]), key % P
        for h in range(t.Hkv):
            raw = pool.view(torch.uint8) if pool.dtype == F8 else pool
            x8 = 0x7F if pool.dtype == F8 else x
            if hnd:
                raw[pg, h, slot, d] = x8
            else:
                raw[pg, slot, h, d] = x8

    put(bad, kv - n + 2, 7, math.inf if t.cache == "bf16" else math.nan)
    put(bad, kv - n + 5, 9, math.nan)
    put(t.k, kv - n + 5, 3, math.nan)
    if t.window >= 0 and kv > 200:
        for key in range(kv - n - t.window):  # no row sees these
            put(bad, key, 0, math.nan)
            put(t.k, key, 0, math.nan)
        gone = (kv - n - t.window) // P
        tail = t.table.clone()
    for key in range(kv, -(-kv // P) * P):
        put(bad, key, 1, math.nan)
        put(t.k, key, 1, math.nan)
    d = t.dev()
    if t.window >= 0 and kv > 200:
        tail[0, :gone] = -1  # pages that were given back
        d["block_tables"] = tail.to(DEV)
    out = cuda_lib.tree_attention(**d)
    assert cuda_lib.device_status() == 0
    fin = torch.isfinite(out).all(-1).all(-1)
    assert set(torch.nonzero(~fin).flatten().tolist()) == {2, 9}
    t.check(out)


def test_a_query_that_is_not_finite_stays_in_its_row(cuda_lib):
    for cache in ("bf16", "e4m3"):
        t = Batch([9], [200], 4, 2, 128, 16, cache=cache)
        clean = cuda_lib.tree_attention(**t.dev())
        t.q[3, 1, 5] = math.nan
        t.q[4, 2, 6] = math.inf
        out = cuda_lib.tree_attention(**t.dev())
        assert torch.isnan(out[3, 1]).all() and torch.isnan(out[4, 2]).all()
        keep = torch.ones((9, 4), dtype=torch.bool)
        keep[3, 1] = keep[4, 2] = False
        assert torch.equal(out[keep.to(DEV)], clean[keep.to(DEV)])


def test_malformed_requests_and_pages(cuda_lib):
    t = Batch([4, 5, 6, 3], [100, 200, 300, 50], 8, 2, 128, 32)
    d = t.dev()
    ref = cuda_lib.tree_attention(**d)
    seq = t.seq.clone()
    seq[1] = 3       # fewer keys than nodes
    seq[2] = 400     # more than max_kv_len
    out = torch.full_like(ref, 9.0)
    for path in ("auto", "generic"):
        cuda_lib.set_kernel_path(path)
        try:
            out.fill_(9.0)
            cuda_lib.tree_attention(**{**d, "seq_lens": seq.to(DEV)}, out=out)
        finally:
            cuda_lib.set_kernel_path("auto")
        assert cuda_lib.device_status() == cuda_lib.DEV_BAD_REQUEST
        assert (out[4:15] == 9).all()
        if path == "auto":
            assert torch.equal(out[:4], ref[:4]) and torch.equal(out[15:], ref[15:])
        # a page id outside the pool: its keys read as K = V = 0
        table = t.table.clone()
        table[0, 1] = t.k.shape[0]
        table[3, 0] = -1
        cuda_lib.set_kernel_path(path)
        try:
            got = cuda_lib.tree_attention(**{**d, "block_tables": table.to(DEV)})
        finally:
            cuda_lib.set_kernel_path("auto")
        assert cuda_lib.device_status() == cuda_lib.DEV_BAD_PAGE
        z = Batch([4, 5, 6, 3], [100, 200, 300, 50], 8, 2, 128, 32)
        for pool in (z.k, z.v):
            pool[int(t.table[0, 1])] = 0
            pool[int(t.table[3, 0])] = 0
        z.check(got)


def test_strides(cuda_lib):
    """Query and output inside wider buffers, one [N, 2, ...] cache, a permuted pool, mask rows apart."""
    t = Batch([6, 10], [150, 90], 8, 2, 128, 16, layout="NHD", seed=2)
    d = t.dev()
    T = t.q.shape[0]
    wide = torch.zeros((T, 8 + 4, 128), dtype=BF, device=DEV)
    wide[:, :8] = d["query"]
    cache = torch.stack([d["kv_cache"][0], d["kv_cache"][1]], 1)  # [N, 2, P, Hkv, D]
    mask = torch.zeros((T, 7), dtype=torch.int32, device=DEV)
    mask[:, 2:3] = d["tree_mask"]
    big = torch.full((8, T + 2, 128), 3.0, dtype=BF, device=DEV)
    out = big.transpose(0, 1)[1:-1]
    cuda_lib.tree_attention(**{**d, "query": wide[:, :8], "kv_cache": cache, "tree_mask": mask[:, 2:3]}, out=out)
    t.check(out)
    assert (big[:, 0] == 3).all() and (big[:, -1] == 3).all()
    perm = tuple(x.transpose(1, 2) for x in d["kv_cache"])  # an HND view of NHD storage
    assert torch.equal(cuda_lib.tree_attention(**{**d, "kv_cache": perm, "kv_layout": "HND"}), out)


def test_workspace_of_the_c_call(cuda_lib):
    """Too little workspace: nothing runs.  Where every tree sees few keys none is needed."""
    import ctypes

    lib = cuda_lib.load()
    for kv, window, small in ((300, -1, True), (512, -1, True), (513, -1, False), (4000, 100, True), (4000, 800, False)):
        t = Batch([5], [kv], 4, 2, 128, 32, window=window)
        d = t.dev()
        out = torch.full_like(d["query"], 3.0)
        need = ctypes.c_uint64(7)

        def call(ws, n):
            return lib.b2pa_tree_attention(
                *(None if x is None else ctypes.byref(cuda_lib.desc(x)) for x in (
                    d["query"], *d["kv_cache"], d["block_tables"], d["seq_lens"], d["cum_seq_lens_q"], d["tree_mask"],
                    d["positions"])),
                5, kv, t.bmm1, t.bmm2, window, None, 0, ctypes.byref(cuda_lib.desc(out)), ws, n, ctypes.byref(need),
                torch.cuda.current_stream().cuda_stream)

        if small:
            assert call(None, 0) == 0 and need.value == 0
        else:
            assert call(None, 0) == -5 and need.value > 0
            ws = torch.empty(need.value, dtype=torch.uint8, device=DEV)
            assert call(ws.data_ptr(), need.value - 1) == -5
            torch.cuda.synchronize()
            assert (out == 3).all()
            assert call(ws.data_ptr(), need.value) == 0
        torch.cuda.synchronize()
        t.check(out)


def test_no_rows(cuda_lib):
    t = Batch([0, 0], [5, 9], 4, 2, 128, 16)
    assert cuda_lib.tree_attention(**t.dev()).shape == (0, 4, 128)


def test_streams_and_two_graphs_at_once(cuda_lib):
    ts = [Batch([9, 12], [3000 + 500 * i, 700], 16, 4, 128, 32, seed=20 + i) for i in range(2)]
    ds = [t.dev() for t in ts]
    ref = [cuda_lib.tree_attention(**d) for d in ds]
    for t, x in zip(ts, ref):
        t.check(x)
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [cuda_lib.tree_attention(**d, stream=s) for d, s in zip(ds, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # two graphs captured on one stream, replayed together on two
    graphs, outs = [], []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cuda_lib.tree_attention(**d))
        graphs.append(g)
    for d, t in zip(ds, ts):
        d["query"].copy_(-t.q.to(DEV))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for t, x in zip(ts, outs):
        t.q = -t.q
        t.check(x)
    assert cuda_lib.device_status() == 0


def test_wait_limit(cuda_lib):
    """A wait that nothing completes runs out: an error bit, and the next call is fine."""
    for name in ("ragged", "two_tiles", "e4m3", "e4m3_two_tiles"):
        t = Batch(**CASES[name])
        d = t.dev()
        ref = cuda_lib.tree_attention(**d)
        torch.cuda.synchronize()
        cuda_lib.set_wait_limit_ns(2_000_000)
        cuda_lib.debug_inject_stall(True)
        try:
            cuda_lib.tree_attention(**d)
        finally:
            cuda_lib.debug_inject_stall(False)
            cuda_lib.set_wait_limit_ns(0)
        assert cuda_lib.device_status() == cuda_lib.DEV_TIMEOUT
        assert torch.equal(cuda_lib.tree_attention(**d), ref)
        assert cuda_lib.device_status() == 0
