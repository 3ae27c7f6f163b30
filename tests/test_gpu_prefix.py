"""Attention of requests that share a cached prefix (b2pa_prefix_attention) on the GPU, against the formula in fp64.

Tolerance, with A = sum p|v| / sum p over the keys a row sees:
  the result's rounding to bf16: 2^-8 |o| (half a step);
  each probability's rounding: to bf16 2^-8 A (over e4m3 caches to f16, 2^-11 A, and 2^-32 p_max sum|v| / sum p for
  those below 2^-21 of the largest);
  scores in fp32 (unit 2^-24, D + 8 roundings of products and sums): ds = 2^-24 (D + 8) bmm1 max_j sum_d |q_d k_jd|,
  over e4m3 caches 2^-17 max|q| bmm1 max_j sum_d |k_jd| more; a score's error changes its weight by that factor, in
  numerator and denominator: 2 ds A;
  the exponent's own rounding and approximation (|x| < 128, 2^-22), and the weights of the merged parts: 2^-15 A."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
BAD_REQUEST, BAD_PAGE, TIMEOUT = 1, 2, 4


def sums(x):
    return [sum(x[:i]) for i in range(len(x) + 1)]


class Batch:
    """Groups of `reqs` requests behind prefixes of `prefix` keys, requests of `ns` tokens and `kvs` own keys; the first
    `alone` requests and the last are in no group where `alone` is given."""

    def __init__(self, reqs, prefix, ns, kvs, H, Hkv, D, P, layout="HND", cache="bf16", sinks=False, seed=0, q_scale=1.0,
                 alone=0):
        g = torch.Generator().manual_seed(seed)
        self.reqs, self.prefix, self.ns, self.kvs = reqs, prefix, ns, kvs
        self.H, self.Hkv, self.D, self.P, self.layout, self.cache = H, Hkv, D, P, layout, cache
        self.starts = [alone + x for x in sums(reqs)]
        shared, own = [-(-x // P) for x in prefix], [-(-x // P) for x in kvs]
        N = sum(shared) + sum(own) + 3
        shape = (N, Hkv, P, D) if layout == "HND" else (N, P, Hkv, D)
        self.k, self.v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        self.bmm1, self.bmm2 = 1 / math.sqrt(D), 1.0
        if cache == "e4m3":
            self.k, self.v = (self.k * 50).to(F8), (self.v * 50).to(F8)
            self.bmm1, self.bmm2 = self.bmm1 / 50, 1 / 50
        else:
            self.k, self.v = self.k.to(BF), self.v.to(BF)
        pages = torch.randperm(N, generator=g).to(torch.int32)
        at = 0

        def table(counts):
            nonlocal at
            t = torch.full((len(counts), max(counts + [0]) + 2), -7, dtype=torch.int32)  # padding is no page
            for b, u in enumerate(counts):
                t[b, :u] = pages[at : at + u]
                at += u
            return t

        self.ptable, self.table = table(shared), table(own)
        # what nobody reads holds NaN: the pages left over, and what lies behind the last keys
        for pg in pages[at:].tolist():
            for pool in (self.k, self.v):
                self.poison(pool[pg])
        for t, lens in ((self.ptable, prefix), (self.table, kvs)):
            for b, n in enumerate(lens):
                if n % P:
                    for pool in (self.k, self.v):
                        x = pool[int(t[b, n // P])]
                        self.poison(x[:, n % P :] if layout == "HND" else x[n % P :])
        self.q = (torch.randn((sum(ns), H, D), generator=g) * q_scale).to(BF)
        self.sinks = torch.randn(H, generator=g) if sinks else None
        self.cum = sums(ns)

    @staticmethod
    def poison(x):
        (x.view(torch.uint8) if x.dtype == F8 else x).fill_(0x7F if x.dtype == F8 else math.nan)

    def group(self, b):
        for g in range(len(self.reqs)):
            if self.starts[g] <= b < self.starts[g + 1]:
                return g
        return None

    def dev(self, **change):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        a = dict(query=self.q.to(DEV), kv_cache=(self.k.to(DEV), self.v.to(DEV)), prefix_tables=self.ptable.to(DEV),
                 prefix_lens=i(self.prefix), cum_groups=i(self.starts), block_tables=self.table.to(DEV),
                 seq_lens=i(self.kvs), max_q_len=max(self.ns + [0]), max_prefix_len=max(self.prefix + [0]),
                 max_kv_len=max(self.kvs + [0]), bmm1_scale=self.bmm1, bmm2_scale=self.bmm2, cum_seq_lens_q=i(self.cum),
                 kv_layout=self.layout, sinks=None if self.sinks is None else self.sinks.to(DEV))
        a.update(change)
        return a

    def rows(self, pool, table, n):
        pg = table[: -(-n // self.P)].long()
        x = pool.view(torch.uint8)[pg].view(F8) if pool.dtype == F8 else pool[pg]
        x = x.to(DEV).to(torch.float64)
        x = x.transpose(1, 2) if self.layout == "HND" else x
        return x.reshape(-1, self.Hkv, self.D)[:n].transpose(0, 1)

    def check(self, out, only=None):
        D, G = self.D, self.H // self.Hkv
        for b, n in enumerate(self.ns):
            if n == 0 or (only is not None and b not in only):
                continue
            g = self.group(b)
            k, v = self.rows(self.k, self.table[b], self.kvs[b]), self.rows(self.v, self.table[b], self.kvs[b])
            pre = 0
            if g is not None:
                pre = self.prefix[g]
                k = torch.cat([self.rows(self.k, self.ptable[g], pre), k], 1)
                v = torch.cat([self.rows(self.v, self.ptable[g], pre), v], 1)
            last = pre + self.kvs[b] - n + torch.arange(n, device=DEV)
            see = (torch.arange(k.shape[1], device=DEV)[None] <= last[:, None]).repeat(G, 1)
            q = self.q[self.cum[b] : self.cum[b] + n].to(DEV).double().transpose(0, 1).reshape(self.Hkv, G * n, D)
            s = torch.where(see, q @ torch.nan_to_num(k).transpose(1, 2) * self.bmm1, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - top)
            den = p.sum(-1, keepdim=True)
            if self.sinks is not None:
                den = den + torch.exp(self.sinks.double().to(DEV).view(self.Hkv, G, 1).repeat_interleave(n, 1) - top)
            fin = torch.isfinite(v)
            v0 = torch.where(fin, v, 0.0)
            o = p @ v0
            if not fin.all():  # what is not finite reaches the rows that see it
                seen = see.double() @ (~fin).double() > 0
                o = torch.where(seen, math.nan, o)
            o = o / den * self.bmm2
            A = (p @ v0.abs()) / den * self.bmm2
            ds = 2.0 ** -24 * (D + 8) * (q.abs() @ torch.nan_to_num(k).abs().transpose(1, 2)).masked_fill(~see, 0).amax(
                -1, keepdim=True) * self.bmm1
            extra = 0.0
            prob = 2.0 ** -8
            if self.cache == "e4m3":
                kmax = torch.nan_to_num(k).abs().sum(-1).amax(-1)[:, None, None]
                ds = ds + 2.0 ** -17 * q.abs().amax(-1, keepdim=True) * kmax * self.bmm1
                extra, prob = 2.0 ** -32 * (see.double() @ v0.abs()) / den * self.bmm2, 2.0 ** -11
            tol = 2.0 ** -8 * o.abs() + A * (prob + 2 * ds + 2.0 ** -15) + extra + 1e-30
            got = out[self.cum[b] : self.cum[b] + n].double().transpose(0, 1).reshape(self.Hkv, G * n, D)
            same = torch.where(torch.isnan(o), ~torch.isfinite(got), (got - o).abs() <= tol)
            assert same.all(), (b, int((~same).sum()), float(torch.nan_to_num((got - o).abs() - tol, nan=9e9).max()))


CASES = {
    "one": dict(reqs=[1], prefix=[1], ns=[1], kvs=[1], H=1, Hkv=1, D=128, P=8),
    "eight_samples": dict(reqs=[8], prefix=[300], ns=[1] * 8, kvs=[1, 2, 31, 32, 33, 64, 5, 9], H=8, Hkv=2, D=128, P=32),
    "two_tiles": dict(reqs=[70], prefix=[1000], ns=[1] * 70, kvs=[1 + i % 40 for i in range(70)], H=8, Hkv=2, D=128, P=16),
    "several_items": dict(reqs=[200], prefix=[700], ns=[1] * 200, kvs=[1 + i % 7 for i in range(200)], H=8, Hkv=2, D=128,
                          P=16),
    "groups": dict(reqs=[3, 1, 0, 9, 33], prefix=[257, 128, 77, 0, 2049], ns=[1] * 46, kvs=[1 + 13 * i for i in range(46)],
                   H=16, Hkv=4, D=128, P=64, layout="NHD", sinks=True),
    "some_alone": dict(reqs=[2, 3], prefix=[500, 129], ns=[1] * 9, kvs=[100, 700, 3, 4, 5, 6, 130, 8, 900], H=8, Hkv=2,
                       D=128, P=32, alone=2),
    "nobody_in_groups": dict(reqs=[], prefix=[], ns=[1, 2], kvs=[300, 2], H=8, Hkv=2, D=128, P=32),
    "chunks": dict(reqs=[3, 2], prefix=[400, 90], ns=[17, 1, 40, 5, 130], kvs=[17, 200, 50, 5, 300], H=8, Hkv=2, D=128,
                   P=16),
    "long_chunks_d64": dict(reqs=[2], prefix=[1500], ns=[300, 280], kvs=[300, 600], H=8, Hkv=1, D=64, P=16, sinks=True),
    "no_tokens": dict(reqs=[4, 1], prefix=[300, 10], ns=[0, 2, 0, 1, 0], kvs=[0, 40, 5, 6, 7], H=4, Hkv=1, D=64, P=8),
    "heads_3": dict(reqs=[30, 14], prefix=[333, 555], ns=[1] * 44, kvs=[9 + i for i in range(44)], H=6, Hkv=2, D=128, P=32),
    "heads_5_d64": dict(reqs=[24, 25], prefix=[333, 100], ns=[1] * 49, kvs=[1 + 3 * i for i in range(49)], H=5, Hkv=1, D=64,
                        P=16),
    "heads_40": dict(reqs=[4, 3], prefix=[333, 200], ns=[1] * 7, kvs=[9] * 7, H=40, Hkv=1, D=128, P=32),
    "heads_128": dict(reqs=[2, 3], prefix=[333, 200], ns=[1, 1, 2, 1, 1], kvs=[40] * 5, H=128, Hkv=1, D=128, P=32),
    "heads_1_d64": dict(reqs=[130, 7], prefix=[1333, 70], ns=[1] * 137, kvs=[1 + i % 9 for i in range(137)], H=4, Hkv=4,
                        D=64, P=8),
    "heads_12": dict(reqs=[3, 14], prefix=[333, 555], ns=[1] * 17, kvs=[9 + 50 * i for i in range(17)], H=24, Hkv=2, D=128,
                     P=32, sinks=True),
    "heads_16_d64": dict(reqs=[30], prefix=[700], ns=[1] * 30, kvs=[1 + 31 * i for i in range(30)], H=16, Hkv=1, D=64, P=16),
    "heads_9_e4m3": dict(reqs=[30, 2], prefix=[700, 3], ns=[1] * 32, kvs=[1 + 31 * i for i in range(32)], H=18, Hkv=2, D=128,
                         P=64, layout="NHD", cache="e4m3"),
    "heads_16_e4m3": dict(reqs=[5], prefix=[300], ns=[1] * 5, kvs=[1, 128, 129, 600, 5], H=16, Hkv=1, D=128, P=16,
                          cache="e4m3", sinks=True),
    "page_256": dict(reqs=[3], prefix=[1000], ns=[1, 2, 1], kvs=[257, 12, 600], H=4, Hkv=1, D=128, P=256),
    "e4m3": dict(reqs=[6, 9], prefix=[700, 300], ns=[1] * 15, kvs=[1 + 40 * i for i in range(15)], H=32, Hkv=8, D=128,
                 P=32, cache="e4m3"),
    "e4m3_two_tiles": dict(reqs=[40, 25], prefix=[900, 130], ns=[1] * 65, kvs=[1 + i for i in range(65)], H=32, Hkv=4,
                           D=128, P=64, layout="NHD", cache="e4m3", sinks=True),
    "e4m3_chunks": dict(reqs=[3], prefix=[900], ns=[20, 1, 33], kvs=[20, 40, 300], H=10, Hkv=2, D=128, P=16, cache="e4m3"),
    "sharp": dict(reqs=[9], prefix=[600], ns=[1] * 9, kvs=[1, 700, 30, 40, 5, 60, 70, 80, 129], H=8, Hkv=2, D=128, P=16,
                  q_scale=8.0),
    # CUDA cores
    "generic_d16": dict(reqs=[2, 3], prefix=[9, 300], ns=[1, 3, 1, 0, 2], kvs=[4, 5, 40, 7, 2], H=4, Hkv=2, D=16, P=4,
                        sinks=True, alone=0),
    "generic_d80_p3": dict(reqs=[3], prefix=[90], ns=[1, 2, 7], kvs=[5, 6, 7], H=6, Hkv=2, D=80, P=3, layout="NHD", alone=1),
    "generic_d256": dict(reqs=[2], prefix=[200], ns=[1, 1], kvs=[33, 1], H=2, Hkv=1, D=256, P=16),
    "generic_e4m3_d64": dict(reqs=[2], prefix=[200], ns=[2, 1], kvs=[77, 9], H=4, Hkv=1, D=64, P=16, cache="e4m3"),
}
CASES["generic_d80_p3"]["reqs"] = [2]  # (the first is in no group)


@pytest.mark.parametrize("hint", [None, 0, "exact"])
@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(cuda_lib, name, hint):
    """With the most tokens of a group known, unknown, and told wrongly."""
    t = Batch(**CASES[name])
    if hint == "exact":
        hint = max([t.cum[b] - t.cum[a] for a, b in zip(t.starts, t.starts[1:])] + [0])
    out = cuda_lib.prefix_attention(**t.dev(max_group_q_len=hint))
    assert cuda_lib.device_status() == 0
    t.check(out)


@pytest.mark.parametrize("name", ["groups", "chunks", "e4m3", "some_alone"])
def test_generic_path_and_padding_rows(cuda_lib, name):
    """The CUDA-core path on tensor-core shapes; rows behind the last request stay as they were; q and out with gaps."""
    t = Batch(**CASES[name])
    T = t.q.shape[0]
    wide = torch.zeros((T + 3, t.H + 2, t.D + 8), dtype=BF, device=DEV)
    q = wide[:, 1 : t.H + 1, : t.D]
    q[:T] = t.q.to(DEV)
    for path in ("auto", "generic"):
        full = torch.full((T + 3, t.H, 2 * t.D), 5.0, dtype=BF, device=DEV)
        out = full[:, :, : t.D]
        cuda_lib.set_kernel_path(path)
        try:
            assert cuda_lib.prefix_attention(**t.dev(query=q), out=out) is out
        finally:
            cuda_lib.set_kernel_path("auto")
        t.check(out)
        assert (out[T:] == 5).all() and (full[:, :, t.D :] == 5).all()
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cache,prefix,own", [("bf16", 70000, 100), ("e4m3", 70000, 100), ("bf16", 100, 70000),
                                              ("bf16", 40000, 40000)])
def test_long_keys_cut_over_all_sms(cuda_lib, cache, prefix, own):
    """The same bits every time."""
    t = Batch([5], [prefix], [1, 1, 2, 1, 1], [own, 3, own, 700, 128], 8, 2, 128, 64, cache=cache, seed=5)
    d = t.dev()
    out = cuda_lib.prefix_attention(**d)
    t.check(out)
    for _ in range(3):
        assert torch.equal(out, cuda_lib.prefix_attention(**d))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cfg", [dict(H=8, Hkv=2, D=128), dict(H=16, Hkv=1, D=128), dict(H=8, Hkv=1, D=64),
                                 dict(H=16, Hkv=1, D=64), dict(H=8, Hkv=1, D=128, cache="e4m3"),
                                 dict(H=15, Hkv=1, D=128, cache="e4m3")], ids=lambda c: "-".join(map(str, c.values())))
@pytest.mark.parametrize("count", [3, 40])
def test_single_tokens_with_long_keys_of_their_own(cuda_lib, cfg, count):
    """Own keys in many parts, beside others of a single key; q 8 times as large in every other request."""
    t = Batch([count], [130], [1] * count, [1 + 9000 * (i % 3 == 0) + 37 * i for i in range(count)], P=32, seed=count, **cfg)
    t.q[::2] *= 8
    d = t.dev()
    out = cuda_lib.prefix_attention(**d)
    t.check(out)
    assert torch.equal(out, cuda_lib.prefix_attention(**d))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 3e4])
def test_queries_small_and_large(cuda_lib, cache, scale):
    """Rows of queries over bf16's range: over e4m3 caches each is scaled to its own f16 range."""
    t = Batch([6], [150], [1] * 6, [40, 1, 200, 7, 130, 64], 16, 2, 128, 16, cache=cache, seed=3)
    t.q = (t.q.double() * scale * torch.tensor([1.0, 2.0 ** -20, 1.0, 2.0 ** -9, 1.0, 1.0])[:, None, None]).to(BF)
    t.check(cuda_lib.prefix_attention(**t.dev()))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("count", [1, 2, 16, 17, 31, 32, 33, 64, 65, 100])
def test_group_sizes(cuda_lib, cache, count):
    """Row counts around those of one and two tiles, few and many requests."""
    t = Batch([count, 1], [1500, 130], [1] * (count + 1), [1 + 37 * i % 300 for i in range(count + 1)], 8, 1, 128, 16,
              cache=cache, sinks=count % 2 == 0, seed=count)
    t.check(cuda_lib.prefix_attention(**t.dev()))
    assert cuda_lib.device_status() == 0


def test_many_requests_and_groups(cuda_lib):
    r = random.Random(1)
    reqs = [r.choice([0, 1, 2, 5, 20]) for _ in range(150)]
    B = sum(reqs) + 6
    ns = [r.choice([0, 1, 1, 1, 3]) for _ in range(B)]
    kvs = [max(n, r.randint(1, 200)) for n in ns]
    t = Batch(reqs, [r.randint(0, 400) for _ in reqs], ns, kvs, 4, 2, 64, 16, seed=6, alone=3)
    t.check(cuda_lib.prefix_attention(**t.dev()))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cache,D", [("bf16", 128), ("e4m3", 128), ("bf16", 64)], ids=["bf16", "e4m3", "d64"])
@pytest.mark.parametrize("sizes", [[0, 1, 2, 5, 20, 40], [0, 1, 2, 5, 16]], ids=["two-tiles", "one-tile"])
@pytest.mark.parametrize("most", [1, 2])
def test_several_requests_per_thread(cuda_lib, cache, D, sizes, most):
    """More requests and groups than threads in a CTA, of a query tile (16 tokens) and of more, with tokens and without."""
    r = random.Random(len(sizes) + most)
    reqs = [r.choice(sizes) for _ in range(160)]
    B = sum(reqs) + 4
    ns = [r.choice([0, 1, 1, most]) for _ in range(B)]
    kvs = [max(n, r.randint(1, 200)) for n in ns]
    t = Batch(reqs, [r.randint(0, 300) for _ in reqs], ns, kvs, 8, 1, D, 32, cache=cache, seed=6, alone=2)
    assert B + 160 > 512
    d, at = t.dev(), [t.cum[b] for b in t.starts]
    t.check(cuda_lib.prefix_attention(**d))
    # told how many tokens a group has at most (one query tile then, where none has more), or fewer than it has
    for count in (max(y - x for x, y in zip(at, at[1:])), 1):
        t.check(cuda_lib.prefix_attention(**d, max_group_q_len=count))
    assert cuda_lib.device_status() == 0


def test_a_shared_prefix_is_the_decode_batch(cuda_lib):
    """The same batch with the prefix's pages in every request's table: both within the bounds of the formula."""
    B, P, pre = 7, 32, 320
    t = Batch([B], [pre], [1] * B, [50, 4, 700, 128, 129, 2000, 1], 16, 4, 128, P, seed=8)
    d = t.dev()
    t.check(cuda_lib.prefix_attention(**d))
    table = torch.cat([d["prefix_tables"][:, : pre // P].expand(B, -1), d["block_tables"].clamp(min=0)], 1).contiguous()
    t.check(cuda_lib.batch_decode(d["query"], d["kv_cache"], table, d["seq_lens"] + pre, 2000 + pre, t.bmm1, t.bmm2))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("path", ["auto", "generic"])
def test_values_that_are_not_finite(cuda_lib, cache, path):
    """NaN in V: in keys of a request's later tokens they reach the rows that see them alone, in the prefix every
    row of its group."""
    t = Batch([3, 2], [200, 140], [12, 1, 40, 3, 1], [12, 30, 300, 9, 200], 8, 2, 128, 16, cache=cache, seed=3)

    def put(table, key, d):
        pg, slot = int(table[key // t.P]), key % t.P
        row = t.v[pg, :, slot]
        (row.view(torch.uint8) if row.dtype == F8 else row)[:, d] = 0x7F if cache == "e4m3" else math.nan

    put(t.table[0], 7, 3)      # rows 7 .. 11 of request 0
    put(t.table[2], 265, 100)  # the later rows of request 2
    put(t.table[2], 299, 5)    # its last row
    put(t.table[4], 199, 64)   # request 4's own key
    cuda_lib.set_kernel_path(path)
    try:
        t.check(cuda_lib.prefix_attention(**t.dev()))
        put(t.ptable[1], 139, 9)  # group 1's prefix
        t.check(cuda_lib.prefix_attention(**t.dev()))
    finally:
        cuda_lib.set_kernel_path("auto")
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("path", ["auto", "generic"])
def test_malformed_requests_and_groups(cuda_lib, path):
    """Their rows stay as they were, and the others are as if they were alone."""
    t = Batch([3, 2, 2], [200, 140, 60], [1, 2, 1, 1, 3, 1, 1], [12, 30, 300, 9, 200, 5, 7], 8, 2, 128, 16, seed=3)
    cuda_lib.set_kernel_path(path)
    try:
        good = cuda_lib.prefix_attention(**t.dev())
        t.check(good)
        for change, skip in ((dict(max_kv_len=299), [2]), (dict(max_q_len=2), [4]), (dict(max_prefix_len=150), [0, 1, 2]),
                             (dict(cum_groups=torch.tensor([0, 3, 5, 8], dtype=torch.int32, device=DEV)), [5, 6]),
                             (dict(cum_groups=torch.tensor([-1, 3, 5, 7], dtype=torch.int32, device=DEV)), [0, 1, 2]),
                             (dict(seq_lens=torch.tensor([12, 1, 300, -4, 200, 5, 7], dtype=torch.int32, device=DEV)), [1, 3]),
                             (dict(prefix_lens=torch.tensor([200, -1, 5000], dtype=torch.int32, device=DEV),
                                   max_prefix_len=9000), [3, 4, 5, 6])):
            out = torch.full_like(good, 5.0)
            cuda_lib.prefix_attention(**t.dev(**change), out=out)
            assert cuda_lib.device_status() == BAD_REQUEST
            for b in range(7):
                rows = slice(t.cum[b], t.cum[b + 1])
                if b in skip:
                    assert (out[rows] == 5).all(), (change, b)
            t.check(out, [b for b in range(7) if b not in skip])
    finally:
        cuda_lib.set_kernel_path("auto")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [(16, 2), (32, 2)], ids=["8-heads", "16-heads"])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("reqs", [[3, 40, 16, 17, 1, 0, 33, 8], [20, 18], [4, 5, 6], [1, 0, 0, 48]],
                         ids=["mixed", "large", "small", "ends"])
def test_groups_of_all_sizes(cuda_lib, cache, heads, n, reqs):
    """Groups of one query tile, of two and of more in one call."""
    g = torch.Generator().manual_seed(11)
    prefix = [0 if x == 0 else int(torch.randint(1, 900, (1,), generator=g)) for x in reqs]
    if len(reqs) > 2:
        prefix[2] = 0
    R = sum(reqs)
    t = Batch(reqs, prefix, [n] * R, torch.randint(n, 300, (R,), generator=g).tolist(), *heads, 128, 32, cache=cache, seed=5)
    t.check(cuda_lib.prefix_attention(**t.dev()))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("heads", [(8, 2), (32, 1)], ids=["one-tile", "two-tiles"])
def test_groups_over_one_another(cuda_lib, heads):
    """cum_groups that fall: flagged, nothing but the groups' rows written, and the next call is right."""
    t = Batch([3, 2, 2], [200, 140, 60], [1] * 7, [12, 30, 300, 9, 200, 5, 7], *heads, 128, 16, seed=3)
    d = t.dev()
    room = torch.full((9, heads[0], 128), 5.0, dtype=torch.bfloat16, device=DEV)
    for groups in ([0, 7, 0, 7], [3, 3, 0, 7]):
        change = dict(cum_groups=torch.tensor(groups, dtype=torch.int32, device=DEV))
        cuda_lib.prefix_attention(**t.dev(**change), out=room[1:8])
        assert cuda_lib.device_status() == BAD_REQUEST
        assert (room[0] == 5).all() and (room[8] == 5).all()
    t.check(cuda_lib.prefix_attention(**d))


@pytest.mark.parametrize("path", ["auto", "generic"])
def test_bad_pages_read_as_zero(cuda_lib, path):
    t = Batch([2, 1], [200, 40], [1, 1, 1], [40, 30, 20], 8, 2, 128, 16, seed=3)
    d = t.dev()
    d["prefix_tables"][0, 3] = t.k.shape[0]
    d["block_tables"][2, 0] = -1
    cuda_lib.set_kernel_path(path)
    try:
        out = cuda_lib.prefix_attention(**d)
    finally:
        cuda_lib.set_kernel_path("auto")
    assert cuda_lib.device_status() == BAD_PAGE
    for pool in (t.k, t.v):
        pool[int(t.ptable[0, 3])] = 0
        pool[int(t.table[2, 0])] = 0
    t.check(out)


@pytest.mark.parametrize("cfg", [dict(H=8, Hkv=2, D=128), dict(H=8, Hkv=1, D=64), dict(H=8, Hkv=2, D=128, cache="e4m3")],
                         ids=["bf16", "d64", "e4m3"])
@pytest.mark.parametrize("count", [3, 60])
def test_wait_limit(cuda_lib, cfg, count):
    """A wait that nothing ends gives up; the next call is right."""
    t = Batch([count], [900], [1] * count, [50] * count, P=16, **cfg)
    d = t.dev()
    cuda_lib.set_wait_limit_ns(2_000_000)
    cuda_lib.debug_inject_stall(True)
    try:
        cuda_lib.prefix_attention(**d)
        assert cuda_lib.device_status() & TIMEOUT
    finally:
        cuda_lib.debug_inject_stall(False)
        cuda_lib.set_wait_limit_ns(0)
    t.check(cuda_lib.prefix_attention(**d))
    assert cuda_lib.device_status() == 0


def test_streams_and_graphs(cuda_lib):
    """Two streams at once; two captured graphs, replayed together on new inputs: each has its own workspace."""
    x = Batch([20, 3], [3000, 100], [1] * 23, [1 + 9 * i for i in range(23)], 16, 4, 128, 32, seed=1)
    y = Batch([20, 3], [3000, 100], [1] * 23, [1 + 9 * i for i in range(23)], 16, 4, 128, 32, seed=2)
    a, b = x.dev(), y.dev()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [cuda_lib.prefix_attention(**z, stream=s) for _ in range(10) for z, s in ((a, streams[0]), (b, streams[1]))]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, outs[i % 2])
    x.check(outs[0])
    y.check(outs[1])
    held = {k: v.clone() for k, v in a.items() if isinstance(v, torch.Tensor)}
    pools = tuple(p.clone() for p in a["kv_cache"])
    call = {**a, **held, "kv_cache": pools}
    graphs, got = [], []
    for s in streams:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            got.append(cuda_lib.prefix_attention(**call))
    for want, args in ((x, a), (y, b)):
        for k, v in held.items():
            v.copy_(args[k])
        for p, src in zip(pools, args["kv_cache"]):
            p.copy_(src)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], got[1])
        want.check(got[0])
    assert cuda_lib.device_status(streams[0]) == 0 and cuda_lib.device_status(streams[1]) == 0
