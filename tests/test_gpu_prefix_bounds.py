"""Prefix attention where the caller's bounds are far from the batch, and where it has very many requests or groups."""
import itertools

import pytest
import torch

from test_gpu_prefix import BF, CASES, DEV, Batch

pytestmark = pytest.mark.gpu
MAX = 2 ** 31 - 257


def spread(t, at, B, empty_groups=0):
    """The calls' arguments with t's requests as requests at[i] of B, the others being empty; and `empty_groups`
    groups without requests before each of t's."""
    ns, kvs = [0] * B, [0] * B
    for i, b in enumerate(at):
        ns[b], kvs[b] = t.ns[i], t.kvs[i]
    where = list(at) + [B]
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table = torch.full((B, t.table.shape[1]), -7, dtype=torch.int32, device=DEV)
    table[torch.tensor(at, device=DEV)] = t.table.to(DEV)
    starts, lens, rows = [], [], []
    for g in range(len(t.reqs)):
        starts += [where[t.starts[g]]] * (empty_groups + 1)
        lens += [0] * empty_groups + [t.prefix[g]]
        rows += [0] * empty_groups + [g]
    starts.append(where[t.starts[-1]])
    return t.dev(block_tables=table, seq_lens=i(kvs), cum_seq_lens_q=i([0] + list(itertools.accumulate(ns))),
                 cum_groups=i(starts), prefix_lens=i(lens), prefix_tables=t.ptable.to(DEV)[torch.tensor(rows, device=DEV)])


@pytest.mark.parametrize("path", ["auto", "generic"])
@pytest.mark.parametrize("name", ["groups", "chunks", "heads_16_e4m3", "some_alone"])
def test_more_requests_than_a_grid_has_rows(cuda_lib, name, path):
    """70000 requests, all but a few of them empty; groups that are empty, too."""
    t = Batch(**CASES[name])
    at = [i * 69999 // (len(t.ns) - 1) for i in range(len(t.ns))]
    d = spread(t, at, 70000, 37)
    out = torch.full(t.q.shape, 5.0, dtype=BF, device=DEV)
    cuda_lib.set_kernel_path(path)
    try:
        t.check(cuda_lib.prefix_attention(**d, out=out))
        assert cuda_lib.device_status() == 0
    finally:
        cuda_lib.set_kernel_path("auto")


@pytest.mark.parametrize("path", ["auto", "generic"])
def test_more_groups_than_requests(cuda_lib, path):
    t = Batch(**CASES["groups"])
    cuda_lib.set_kernel_path(path)
    try:
        t.check(cuda_lib.prefix_attention(**spread(t, range(len(t.ns)), len(t.ns), 3000)))
        assert cuda_lib.device_status() == 0
    finally:
        cuda_lib.set_kernel_path("auto")


@pytest.mark.parametrize("name", ["one", "eight_samples", "groups", "chunks", "some_alone", "nobody_in_groups", "no_tokens",
                                  "heads_16_d64", "heads_16_e4m3", "e4m3_two_tiles", "e4m3_chunks", "generic_d80_p3"])
@pytest.mark.parametrize("bounds", [dict(max_q_len=4096), dict(max_q_len=2 ** 31 - 1, max_prefix_len=MAX, max_kv_len=MAX),
                                    dict(max_prefix_len=MAX), dict(max_kv_len=MAX)],
                         ids=["tokens", "all", "prefix", "own"])
def test_loose_bounds(cuda_lib, name, bounds):
    t = Batch(**CASES[name])
    t.check(cuda_lib.prefix_attention(**t.dev(**bounds)))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cfg", [dict(H=8, Hkv=2, D=128), dict(H=8, Hkv=2, D=64), dict(H=8, Hkv=2, D=128, cache="e4m3"),
                                 dict(H=32, Hkv=2, D=128), dict(H=32, Hkv=2, D=64), dict(H=24, Hkv=2, D=128, cache="e4m3")],
                         ids=lambda c: "-".join(map(str, c.values())))
@pytest.mark.parametrize("kind", ["two-tiles", "one-tile", "short-requests"])
@pytest.mark.parametrize("over", [False, True], ids=["below", "above"])
def test_steps_at_the_limit_of_32_bits(cuda_lib, cfg, kind, over):
    """Bounds on the lengths for which the steps of all units just fit 2e9, and for which they do not."""
    G = cfg["H"] // cfg["Hkv"]
    tile = 4 * (32 // G)  # tokens of a query tile
    reqs = [tile] * 5 + [3] * 30 if kind == "one-tile" else [tile + 9, 2 * tile + 1] + [1] * 60
    n = 3 if kind == "short-requests" else 1
    B = sum(reqs)
    t = Batch(reqs, [1 + 31 * g % 500 for g in range(len(reqs))], [n] * B, [n + 41 * b % 300 for b in range(B)], P=32, seed=2,
              **cfg)
    units = (len(reqs) * (n * B // tile + 1) + B) * cfg["Hkv"]
    steps = int(2e9) // units
    assert units * (MAX // 128 + 5) >= 2e9 > units * steps // 2
    bound = MAX if over else (steps - 6) * 128
    d = t.dev(max_prefix_len=bound, max_kv_len=bound)
    at = [t.cum[b] for b in t.starts]
    most = max(y - x for x, y in zip(at, at[1:]))
    out = cuda_lib.prefix_attention(**d, max_group_q_len=most)
    t.check(out)
    assert cuda_lib.device_status() == 0
    t.check(cuda_lib.prefix_attention(**t.dev(), max_group_q_len=most))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_long_chunk_beside_single_tokens(cuda_lib, cache):
    t = Batch([40, 21], [500, 130], [1] * 30 + [700] + [1] * 30, [1 + 7 * b for b in range(30)] + [900] + [30] * 30, 8, 2, 128,
              32, cache=cache, seed=3)
    t.check(cuda_lib.prefix_attention(**t.dev()))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("first", [100, -3, 0, 10])
def test_requests_beside_offsets_that_fall(cuda_lib, cache, first):
    """One start of cum_q that is none: the two requests that it bounds are malformed, or empty; the others are served,
    and tokens that nobody owns stay as they were."""
    t = Batch([3, 2, 2], [200, 140, 60], [1, 2, 1, 1, 3, 1, 1], [12, 30, 300, 9, 200, 5, 7], 8, 2, 128, 16, cache=cache,
              seed=3)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    d = t.dev()
    # requests 2 and 3 of eight are [3, first) and [first, 4); request 2 of t is neither
    q = torch.cat([d["query"], d["query"][:2]])
    rows = torch.tensor([0, 1, 2, 2, 3, 4, 5, 6], device=DEV)
    d.update(query=q, cum_seq_lens_q=i([0, 1, 3, first, 4, 5, 8, 9, 10]), block_tables=d["block_tables"][rows],
             seq_lens=i([12, 30, 1, 1, 9, 200, 5, 7]), cum_groups=i([0, 4, 6, 8]))
    out = torch.full(q.shape, 5.0, dtype=BF, device=DEV)
    cuda_lib.prefix_attention(**d, out=out)
    assert cuda_lib.device_status() == 1  # BAD_REQUEST
    assert (out[3] == 5).all() and (out[10:] == 5).all()
    t.check(out, [0, 1, 3, 4, 5, 6])


@pytest.mark.parametrize("length", [96, 100, 127, 64])
def test_rows_of_a_ledger(cuda_lib, length):
    """A prompt forked to neighbouring rows, which grow: the prefix and the own keys are views of the ledger's rows."""
    P, R, N, pre = 32, 6, 40, length // 32
    g = torch.Generator(device=DEV).manual_seed(length)
    pools = tuple(torch.randn((N, 2, P, 128), generator=g, device=DEV).to(BF) for _ in "kv")
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table, seq, refs = torch.zeros((R, 12), dtype=torch.int32, device=DEV), i([0] * R), i([0] * N)
    cuda_lib.grow_pages(table, seq, refs, i([0]), i([length]), P)
    src, dst = cuda_lib.fork_pages(table, seq, refs, i([0] * 4), i([1, 2, 3, 4]), P)
    cuda_lib.copy_pages(pools, src, dst)
    cuda_lib.grow_pages(table, seq, refs, i([1, 2, 3, 4]), seq[1:5] + i([1, 40, 33, 7]), P)
    assert cuda_lib.device_status() == 0
    q = torch.randn((4, 8, 128), generator=g, device=DEV).to(BF)
    out = cuda_lib.prefix_attention(q, pools, table[:1, :pre], i([pre * P]), i([0, 4]), table[1:5, pre:],
                                    seq[1:5] - pre * P, 1, pre * P, 4 * P, 128 ** -0.5, 1.0, i([0, 1, 2, 3, 4]))
    assert cuda_lib.device_status() == 0
    rows, lens = table.tolist(), seq.tolist()
    for b in range(4):
        k, v = (x[rows[1 + b][: -(-lens[1 + b] // P)]].transpose(0, 1).reshape(2, -1, 128)[:, : lens[1 + b]].double()
                for x in pools)
        x = q[b].double().view(2, 4, 128)
        p = torch.softmax(x @ k.transpose(1, 2) * 128 ** -0.5, -1)
        want, mean = (p @ v).view(8, 128), (p @ v.abs()).view(8, 128)
        # bf16's half step of the result, of each probability, and what is in 32 bits (see test_gpu_prefix.py)
        ds = 2.0 ** -24 * 136 * (x.abs() @ k.abs().transpose(1, 2)).amax() * 128 ** -0.5
        assert ((out[b].double() - want).abs() <= 2.0 ** -8 * want.abs() + mean * (2.0 ** -8 + 2 * ds + 2.0 ** -15)).all()
