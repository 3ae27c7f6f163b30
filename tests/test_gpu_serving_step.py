"""The calls of a serving step one after the other, as an engine makes them:
queries and keys normed and rotated inside the projection's output, keys and
values written to the pools, drafted trees attended to; and a prefix kept in
the scaled e4m3 cache, restored into bf16 pages and attended to.  Each step is
compared with plain torch on what the step before it really gave, so that every
tolerance is one step's own (bf16's half step is 2^-8)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
H, HK, D, P = 8, 2, 128, 16


def table(n):
    inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


def rotated(x, w, cs, pos):
    x = x.double()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    c, s = cs.double()[pos.long(), : D // 2][:, None], cs.double()[pos.long(), D // 2 :][:, None]
    a, b = x[..., : D // 2], x[..., D // 2 :]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def attend(q, k, v, see):
    """q [n, H, D], k / v [kv, HK, D] in fp64, see [n, kv]: (out, sum p|v| / sum p)."""
    k, v = (x.double().repeat_interleave(H // HK, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", q.double(), k) / math.sqrt(D)
    p = torch.softmax(torch.where(see, s, -math.inf), -1)
    return torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())


def near(got, ref, size, n):
    """Within n half steps of bf16 of `size`, and one of the result."""
    assert ((got.double() - ref).abs() <= 2.0 ** -8 * (n * size + ref.abs()) + 1e-6).all()


def test_draft_and_verify(cuda_lib):
    """Two rounds: a prompt prefilled, then a drafted tree verified, the second time from a captured graph."""
    b2pa = cuda_lib
    g = torch.Generator(device=DEV).manual_seed(3)
    lens, nodes = [70, 33, 128], [6, 9, 1]
    B, cs = 3, table(400)
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(BF) for _ in "qk")
    N = 40
    kp, vp = (torch.full((N, HK, P, D), math.nan, dtype=BF, device=DEV) for _ in "kv")
    pages = torch.randperm(N, generator=g, device=DEV)[: B * 12].view(B, 12).to(torch.int32)

    def slots(b, pos):
        return pages[b].long()[pos // P] * P + pos % P

    def step(qkv, pos, loc):
        """Norm and rotation in place, and the write; returns (q, k, v) views."""
        T = qkv.shape[0]
        q, k = qkv[:, : H * D].view(T, H, D), qkv[:, H * D : (H + HK) * D].view(T, HK, D)
        v = qkv[:, (H + HK) * D :].view(T, HK, D)
        b2pa.qk_norm_rope(q, k, cs, pos, qw, kw, q_out=q, k_out=k)
        b2pa.append_kv(k, v, (kp, vp), loc)
        return q, k, v

    def project(T):
        return torch.randn((T, (H + 2 * HK) * D), generator=g, device=DEV).to(BF)

    # the prompts
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).to(DEV)
    loc = torch.cat([slots(b, torch.arange(n, device=DEV)) for b, n in enumerate(lens)]).to(torch.int32)
    raw = project(sum(lens))
    before = raw.clone()
    q, k, v = step(raw, pos, loc)
    near(q, rotated(before[:, : H * D].view(-1, H, D), qw, cs, pos), 0, 0)
    cum = torch.tensor([0, 70, 103, 231], dtype=torch.int32, device=DEV)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = b2pa.context_attention(q, (kp, vp), pages, seq, 128, 128, 1 / math.sqrt(D), 1.0, cum)
    keys = [k[int(cum[b]) : int(cum[b + 1])].clone() for b in range(B)]
    vals = [v[int(cum[b]) : int(cum[b + 1])].clone() for b in range(B)]
    for b, n in enumerate(lens):
        see = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
        near(out[int(cum[b]) : int(cum[b + 1])], *attend(q[int(cum[b]) : int(cum[b + 1])], keys[b], vals[b], see), 2)

    # trees on top of them: parent of node i is i - 2, or the prompt's last token
    T = sum(nodes)
    masks, depth = [], []
    for n in nodes:
        m = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            if i >= 2:
                m[i] = m[i - 2]
            m[i, i] = True
        masks.append(m)
        depth += (m.sum(1) - 1).tolist()
    words = torch.cat([(m.long() << torch.arange(m.shape[0])).sum(1) for m in masks])[:, None].to(torch.int32).to(DEV)
    ctx = torch.cat([torch.full((n,), x) for n, x in zip(nodes, lens)])
    tree_pos = (ctx + torch.tensor(depth)).to(torch.int32).to(DEV)
    place = torch.cat([slots(b, lens[b] + torch.arange(n, device=DEV)) for b, n in enumerate(nodes)]).to(torch.int32)
    tree_cum = torch.tensor([0, 6, 15, 16], dtype=torch.int32, device=DEV)
    tree_seq = torch.tensor([a + b for a, b in zip(lens, nodes)], dtype=torch.int32, device=DEV)
    qkv = project(T)

    def verify():
        tq, tk, tv = step(qkv, tree_pos, place)
        return tq, tk, tv, b2pa.tree_attention(tq, (kp, vp), pages, tree_seq, words, 9, 140, 1 / math.sqrt(D), 1.0,
                                               tree_cum)

    def check(raw, tq, tk, tv, out):
        near(tq, rotated(raw[:, : H * D].view(-1, H, D), qw, cs, tree_pos), 0, 0)
        near(tk, rotated(raw[:, H * D : (H + HK) * D].view(-1, HK, D), kw, cs, tree_pos), 0, 0)
        for b, (n, m) in enumerate(zip(nodes, masks)):
            lo, hi = int(tree_cum[b]), int(tree_cum[b + 1])
            see = torch.cat([torch.ones((n, lens[b]), dtype=torch.bool), m], 1).to(DEV)
            near(out[lo:hi], *attend(tq[lo:hi], torch.cat([keys[b], tk[lo:hi]]), torch.cat([vals[b], tv[lo:hi]]), see), 2)

    raw = qkv.clone()
    check(raw, *verify())
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # append_kv wants one call on a stream before its capture
        verify()
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        held = verify()
    for _ in range(2):
        raw = project(T)
        qkv.copy_(raw)
        graph.replay()
        torch.cuda.synchronize()
        check(raw, *held)
    assert b2pa.device_status() == 0 and b2pa.device_status(side) == 0


def test_prefix_from_the_scaled_cache(cuda_lib):
    """A prefix quantised row by row, restored into pages of bf16 pools, and read by both attentions."""
    b2pa = cuda_lib
    g = torch.Generator(device=DEV).manual_seed(5)
    n, new = 150, 5
    k = torch.randn((n + new, HK, D), generator=g, device=DEV) * torch.exp2(torch.randn((n + new, HK, 1), generator=g, device=DEV))
    k, v = k.to(BF), torch.randn((n + new, HK, D), generator=g, device=DEV).to(BF)
    store = tuple(torch.zeros((12, P, HK, D), dtype=torch.uint8, device=DEV).view(F8) for _ in "kv")
    scales = tuple(torch.zeros((12, P, HK), device=DEV) for _ in "kv")
    loc = torch.randperm(12 * P, generator=g, device=DEV)[:n].to(torch.int32)
    b2pa.append_kv_scaled(k[:n], v[:n], store, scales, loc, kv_layout="NHD")
    # pages of the working pools, in order: rows 0 .. n - 1 of a flat view
    kp, vp = (torch.zeros((12, P, HK, D), dtype=BF, device=DEV) for _ in "kv")
    rows = [x.view(12 * P, HK, D) for x in (kp, vp)]
    b2pa.read_kv_scaled(store, scales, loc, k_out=rows[0][:n], v_out=rows[1][:n], kv_layout="NHD")
    for got, x in ((rows[0][:n], k[:n]), (rows[1][:n], v[:n])):
        # half an e4m3 step is 2^-4 of a value, and 2^-10 scales at the least, a scale being at most 2^-7.8 of the
        # row's largest value
        assert ((got.double() - x.double()).abs() <= x.double().abs() * 2.0 ** -4
                + 2.0 ** -17 * x.double().abs().amax(-1, keepdim=True)).all()
    b2pa.append_kv(k[n:], v[n:], (kp, vp), torch.arange(n, n + new, dtype=torch.int32, device=DEV), kv_layout="NHD")
    q = torch.randn((new, H, D), generator=g, device=DEV).to(BF)
    seq = torch.tensor([n + new], dtype=torch.int32, device=DEV)
    cum = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    pages = torch.arange(12, dtype=torch.int32, device=DEV)[None]
    see = torch.ones((new, n + new), dtype=torch.bool, device=DEV).tril(n)
    chain = torch.tensor([[(1 << (i + 1)) - 1] for i in range(new)], dtype=torch.int32, device=DEV)
    ref = attend(q, rows[0][: n + new], rows[1][: n + new], see)
    near(b2pa.context_attention(q, (kp, vp), pages, seq, new, n + new, 1 / math.sqrt(D), 1.0, cum, kv_layout="NHD"), *ref, 2)
    near(b2pa.tree_attention(q, (kp, vp), pages, seq, chain, new, n + new, 1 / math.sqrt(D), 1.0, cum, kv_layout="NHD"),
         *ref, 2)
    assert b2pa.device_status() == 0


def test_calls_from_several_threads(cuda_lib):
    """Host threads with a stream each, the same tensors read by all."""
    import threading

    b2pa = cuda_lib
    g = torch.Generator(device=DEV).manual_seed(8)
    kp, vp = (torch.randn((30, HK, P, D), generator=g, device=DEV).to(BF) for _ in "kv")
    q = torch.randn((7, H, D), generator=g, device=DEV).to(BF)
    args = (q, (kp, vp), torch.arange(30, dtype=torch.int32, device=DEV)[None],
            torch.tensor([470], dtype=torch.int32, device=DEV),
            torch.tensor([[(1 << (i + 1)) - 1] for i in range(7)], dtype=torch.int32, device=DEV), 7, 470,
            1 / math.sqrt(D), 1.0, torch.tensor([0, 7], dtype=torch.int32, device=DEV))
    ref = b2pa.tree_attention(*args)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(30):
            x = b2pa.tree_attention(*args, stream=s)
            s.synchronize()
            if not torch.equal(x, ref):
                bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
