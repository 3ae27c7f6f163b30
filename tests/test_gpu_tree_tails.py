"""Tree attention over an e4m3 cache where one key leads each row and a long, low tail follows it, as a row that
rests on a sink token has: the tail's probabilities are small one by one and heavy together.  Against the formula
in fp64, with values whose mean is not 0, so that a lost or a rounded-up tail shows.

Tolerance, with A = sum p|v| / sum p:
  the result's rounding to bf16: 2^-8 |o| (half a step);
  each probability's rounding to f16: 2^-11 A, and where f16 has no normal value any more half a step of 2^-24,
  the row's largest being at 2^7 or more: 2^-32 p_max sum|v| / sum p (2^-16 |v| at 65536 keys);
  scores: fp32 products and sums, 2^-24 (D + 8) bmm1 max_j sum_d |q_d k_jd|, and q in two e4m3 terms, 2^-17
  max|q| bmm1 max_j sum_d |k_jd|; each changes a weight by that factor, above and below the line: 2 ds A;
  the exponent's own rounding and approximation: 2^-15 A."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
D, P = 128, 32

# nodes, query heads per kv head: 32, 64, 100, 128 and 256 rows of a kv head
SHAPES = {"rows_1": (1, 1), "rows_32": (8, 4), "rows_64": (16, 4), "rows_100": (25, 4), "rows_128": (4, 32),
          "two_tiles": (64, 4)}


def make(ns, kvs, G, lead, spread, values, seed=0, Hkv=2):
    """One e4m3 batch: key 0 of every request scores `lead` nats over the rest, whose scores deviate by `spread`."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    used = [-(-k // P) for k in kvs]
    N = sum(used) + 2
    # q is 1 in the first column and small multiples of 2^-6 in the others; the first column of K carries the lead
    q = torch.randint(-16, 17, (sum(ns), G * Hkv, D), generator=g, device=DEV).float() / 64
    q[..., 0] = 1.0
    rms = math.sqrt((D - 1) * (sum(i * i for i in range(-16, 17)) / 33)) / 64  # of a product with unit keys
    bmm1 = max(lead, 1e-3) / 256
    k = torch.randn((N, Hkv, P, D), generator=g, device=DEV) * (spread / bmm1 / rms)
    k[..., 0] = 0
    if values == "ones":
        v = torch.ones((N, Hkv, P, D), device=DEV)
    else:
        v = 0.3 + 0.1 * torch.randn((N, Hkv, P, D), generator=g, device=DEV)
    table = torch.full((len(kvs), max(used)), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(N, generator=g, device=DEV).to(torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at : at + u]
        at += u
        first = int(order[at - u])
        k[first, :, 0] = 0
        k[first, :, 0, 0] = 256.0
        if values != "ones":
            v[first, :, 0] = 2.0 ** -6
    k, v = k.clamp(-448, 448).to(F8), v.to(F8)
    cum = [sum(ns[:i]) for i in range(len(ns) + 1)]
    words = max(1, -(-max(ns) // 32))
    chain = torch.zeros((sum(ns), words), dtype=torch.int64)
    for b, n in enumerate(ns):
        for i in range(n):
            for j in range(i + 1):
                chain[cum[b] + i, j // 32] |= 1 << (j % 32)
    chain = torch.where(chain >= 1 << 31, chain - (1 << 32), chain).to(torch.int32)
    args = dict(query=q.to(BF), kv_cache=(k, v), block_tables=table,
                seq_lens=torch.tensor(kvs, dtype=torch.int32, device=DEV), tree_mask=chain.to(DEV), max_q_len=max(ns),
                max_kv_len=max(kvs), bmm1_scale=bmm1, bmm2_scale=1.0,
                cum_seq_lens_q=torch.tensor(cum, dtype=torch.int32, device=DEV))
    return args, ns, kvs, G, Hkv


def check(case, out, p_small=2.0 ** -32):
    args, ns, kvs, G, Hkv = case
    row = 0
    for b, (n, kv) in enumerate(zip(ns, kvs)):
        pages = args["block_tables"][b, : -(-kv // P)].long()
        k, v = (x.view(torch.uint8)[pages].view(F8).to(torch.float64).transpose(0, 1).reshape(Hkv, -1, D)[:, :kv]
                for x in args["kv_cache"])
        q = args["query"][row : row + n].double().transpose(0, 1).reshape(Hkv, G * n, D)
        i, j = torch.arange(n, device=DEV), torch.arange(kv, device=DEV)
        see = (j[None] <= (kv - n + i)[:, None]).repeat(G, 1)
        s = (q @ k.transpose(1, 2) * args["bmm1_scale"]).masked_fill(~see, -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        den = p.sum(-1, keepdim=True)
        o = (p @ v) / den
        A = (p @ v.abs()) / den
        big = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True)
        ds = args["bmm1_scale"] * (2.0 ** -24 * (D + 8) * big + 2.0 ** -17 * q.abs().amax(-1, keepdim=True)
                                   * k.abs().sum(-1).amax(-1)[:, None, None])
        tol = 2.0 ** -8 * o.abs() + A * (2.0 ** -11 + 2 * ds + 2.0 ** -15) + p_small * (see.double() @ v.abs()) / den
        got = out[row : row + n].double().transpose(0, 1).reshape(Hkv, G * n, D)
        off = (got - o).abs()
        assert (off <= tol).all(), (b, float((off / tol).max()), float((off / o.abs()).max()))
        row += n


@pytest.mark.parametrize("keys", [2048, 16384, 65536])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lead", [8.0, 9.5, 11.0, 14.0])
def test_equal_values_come_back(cuda_lib, shape, keys, lead):
    """V = 1 everywhere and equal keys behind the lead: the result is 1 whatever the weights are."""
    n, G = SHAPES[shape]
    case = make([n], [keys], G, lead, 0.0, "ones")
    out = cuda_lib.tree_attention(**case[0])
    assert cuda_lib.device_status() == 0
    check(case, out)


@pytest.mark.parametrize("keys", [4096, 16384, 65536])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lead", [6.0, 8.0, 10.0, 11.0, 14.0])
def test_a_tail_keeps_its_weight(cuda_lib, shape, keys, lead):
    n, G = SHAPES[shape]
    case = make([n], [keys], G, lead, 0.5, "mean", seed=int(lead) + keys)
    out = cuda_lib.tree_attention(**case[0])
    assert cuda_lib.device_status() == 0
    check(case, out)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kvs", [[512] * 24, [1024] * 10, [300, 5000, 80, 2100] * 4], ids=lambda k: f"{len(k)}x{k[0]}")
def test_batches_whole_and_cut(cuda_lib, shape, kvs):
    n, G = SHAPES[shape]
    for lead, spread, values in ((7.0, 0.0, "ones"), (9.0, 0.5, "mean")):
        case = make([n] * len(kvs), kvs, G, lead, spread, values, seed=len(kvs))
        check(case, cuda_lib.tree_attention(**case[0]))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("shape", ["rows_32", "rows_100", "two_tiles"])
@pytest.mark.parametrize("lead,spread,values", [(9.5, 0.0, "ones"), (10.0, 0.0, "ones"), (11.0, 0.5, "mean")])
def test_a_unit_to_an_sm(cuda_lib, shape, lead, spread, values):
    """As many units as SMs: a tail of 16384 keys in one piece behind its lead."""
    n, G = SHAPES[shape]
    case = make([n] * 76, [16384] * 76, G, lead, spread, values, seed=2)
    check(case, cuda_lib.tree_attention(**case[0]))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("lead", [8.0, 11.0, 14.0])
@pytest.mark.parametrize("keys", [4096, 65536])
def test_a_chain_is_the_decode_batch_over_e4m3(cuda_lib, keys, lead):
    """Verifying a drafted chain and decoding over one e4m3 cache: both within the bounds of the formula.  (The decode
    kernel's largest P is 1 or more: its smallest f16 steps weigh 2^-25 of that.)"""
    n, G = 4, 4
    case = make([n] * 3, [keys, 700, keys // 2], G, lead, 0.5, "mean", seed=3)
    d = case[0]
    check(case, cuda_lib.tree_attention(**d))
    ref = cuda_lib.batch_decode(d["query"], d["kv_cache"], d["block_tables"].clamp(min=0), d["seq_lens"], keys,
                                d["bmm1_scale"], 1.0, q_len_per_req=n)
    check(case, ref, p_small=2.0 ** -25)


@pytest.mark.parametrize("shape", ["rows_32", "rows_100", "two_tiles"])
def test_the_same_bits_every_time(cuda_lib, shape):
    """Long and short requests, many calls: what a ring entry holds is read before its next tile comes."""
    n, G = SHAPES[shape]
    kvs = [max(n, k) for k in [100, 500, 1000, 1100, 9000, 4] * 5]
    case = make([n] * len(kvs), kvs, G, 5.0, 1.0, "mean", seed=9)
    first = cuda_lib.tree_attention(**case[0])
    check(case, first)
    for _ in range(10):
        outs = [cuda_lib.tree_attention(**case[0]) for _ in range(40)]
        assert all(torch.equal(x, first) for x in outs)
    assert cuda_lib.device_status() == 0


def test_two_streams_and_two_graphs_at_once(cuda_lib):
    """Calls over one e4m3 cache each, at the same time on two streams, then replayed from two graphs with other queries."""
    cases = [make([8, 3, 0, 6], [9000, 700, 40, 2000 + i], 4, 9.0, 0.5, "mean", seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [cuda_lib.tree_attention(**c[0], stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for c, x in zip(cases, got):
        check(c, x)
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cuda_lib.tree_attention(**c[0]))
        graphs.append(g)
    for c in cases:
        c[0]["query"].copy_(c[0]["query"].flip(0))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, x in zip(cases, outs):
        check(c, x)
    assert cuda_lib.device_status() == 0
