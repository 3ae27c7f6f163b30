"""Query/key norm and rotation (b2pa_qk_norm_rope) on the GPU against the
formula in fp64: pairings, rotary widths, several position axes, strided and
in-place rows, weights, positions outside the table, streams and graphs.

Tolerance: the result is rounded to bf16 once (half a step, 2^-8 of the
value).  Before that, in fp32 (unit 2^-24): the sum of squares goes through at
most 16 + 4 additions of positive terms (20 units, half of them after the
root), the division, eps, the root (2 ulp), weight and product at most 10, the
rotation 3, all relative to |a| + |b| of the pair: under 32 units of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def table(max_pos, R):
    inv = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / R)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def want(x, w, cos_sin, pos, axis_of, interleaved, eps):
    """(value, size of its pair) in fp64."""
    x = x.double()
    half = cos_sin.shape[1] // 2
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    pos = pos.long().view(-1, x.shape[0])
    ax = torch.tensor(axis_of if axis_of is not None else [0] * half)
    i = torch.arange(half)
    at = pos[ax].t()  # [T, half]
    c, s = cos_sin.double()[at, i][:, None], cos_sin.double()[at, half + i][:, None]
    y, size = x.clone(), x.abs()
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def check(got, ref):
    y, size = ref
    err = (got.cpu().double() - y).abs()
    tol = y.abs() * 2.0 ** -8 + size * 32 * 2.0 ** -24 + 2.0 ** -133
    assert (err <= tol).all(), (err - tol).max()


CASES = [
    # T, H, Hkv, D, R, axes, interleaved, weights
    (1, 1, 1, 8, 2, 1, False, "bf16"),
    (1, 32, 8, 128, 128, 1, False, "bf16"),
    (33, 32, 8, 128, 128, 1, False, "fp32"),
    (700, 32, 8, 128, 128, 1, False, "bf16"),  # several rows per group
    (257, 5, 3, 128, 64, 1, False, "bf16"),    # partial rotation, heads not a multiple of four
    (129, 6, 2, 64, 64, 1, True, "bf16"),
    (900, 7, 5, 64, 32, 1, True, "none"),
    (65, 4, 1, 80, 80, 1, False, "bf16"),      # halves that are not whole chunks of lanes
    (65, 4, 1, 80, 40, 1, False, "fp32"),
    (3000, 4, 4, 80, 40, 1, False, "bf16"),
    (65, 4, 1, 80, 50, 1, True, "bf16"),
    (65, 3, 1, 96, 96, 2, False, "bf16"),
    (64, 8, 2, 128, 128, 3, False, "bf16"),
    (64, 8, 2, 128, 128, 3, True, "none"),
    (31, 2, 1, 256, 256, 4, False, "fp32"),
    (1200, 8, 8, 256, 128, 1, True, "bf16"),
    (50, 3, 2, 72, 72, 2, False, "bf16"),
    (50, 3, 2, 104, 16, 1, False, "none"),
    (40, 1, 9, 248, 242, 1, False, "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_formula(cuda_lib, case):
    T, H, K, D, R, axes, inter, weights = case
    g = torch.Generator().manual_seed(7 + CASES.index(case))
    qkv = (torch.randn((T, (H + 2 * K) * D), generator=g) * 3).to(BF)
    q, k = qkv[:, : H * D].view(T, H, D), qkv[:, H * D : (H + K) * D].view(T, K, D)
    w = [None, None]
    if weights != "none":
        w = [(1 + torch.randn(D, generator=g) * 0.3).to(BF if weights == "bf16" else torch.float32) for _ in w]
    cs = table(5000, R)
    pos = torch.randint(0, 5000, (axes, T), generator=g, dtype=torch.int32)
    # frequencies dealt to the axes in turn (no eight in a row alike) or in blocks
    axis_of = None if axes == 1 else [i % axes for i in range(R // 2)] if inter else [
        min(axes - 1, i * axes // (R // 2)) for i in range(R // 2)]
    d = qkv.to(DEV)
    dq, dk = d[:, : H * D].view(T, H, D), d[:, H * D : (H + K) * D].view(T, K, D)
    dw = [None if x is None else x.to(DEV) for x in w]
    qo, ko = cuda_lib.qk_norm_rope(dq, dk, cs.to(DEV), (pos if axes > 1 else pos[0]).to(DEV), *dw, eps=1e-5,
                                   axis_of=axis_of, interleaved=inter)
    assert cuda_lib.device_status() == 0
    check(qo, want(q, w[0], cs, pos, axis_of, inter, 1e-5))
    check(ko, want(k, w[1], cs, pos, axis_of, inter, 1e-5))
    assert torch.equal(d.cpu(), qkv)  # inputs as they were
    # in place, inside the projection's output: the same bits, nothing else touched
    cuda_lib.qk_norm_rope(dq, dk, cs.to(DEV), pos.to(DEV), *dw, eps=1e-5,
                          axis_of=axis_of, interleaved=inter, q_out=dq, k_out=dk)
    assert torch.equal(dq, qo) and torch.equal(dk, ko)
    assert torch.equal(d[:, (H + K) * D :].cpu(), qkv[:, (H + K) * D :])


@pytest.mark.parametrize("case", [
    (13000, 1, 1, 128, 128, 1, False, "bf16"),  # two sets per token
    (6100, 3, 1, 128, 64, 3, False, "fp32"),    # axes in blocks, partial rotation
    (9000, 5, 1, 64, 64, 2, True, "none"),      # axes in turn
    (4000, 4, 3, 128, 50, 1, True, "bf16"),     # pairs that end inside a lane
    (2500, 6, 2, 256, 256, 4, False, "fp32"),
    (1, 20000, 9000, 128, 128, 1, False, "bf16"),  # one token for all
], ids=lambda c: "-".join(map(str, c)))
def test_many_rows(cuda_lib, case):
    """Enough rows for the kernel that goes through them in runs; some positions are outside the table."""
    T, H, K, D, R, axes, inter, weights = case
    g = torch.Generator().manual_seed(T)
    q, k = torch.randn((T, H, D), generator=g).to(BF), torch.randn((T, K, D), generator=g).to(BF)
    w = [None, None]
    if weights != "none":
        w = [(1 + torch.randn(D, generator=g) * 0.3).to(BF if weights == "bf16" else torch.float32) for _ in w]
    cs = table(300, R)
    pos = torch.randint(0, 300, (axes, T), generator=g, dtype=torch.int32)
    axis_of = None if axes == 1 else [i % axes if inter else min(axes - 1, i * axes // (R // 2)) for i in range(R // 2)]
    bad = torch.zeros(T, dtype=torch.bool)
    for t in range(5, T, 97):
        pos[t % axes, t] = -1 if t % 2 else 300
        bad[t] = True
    out = torch.full((T, H, D), 5.0, dtype=BF, device=DEV), torch.full((T, K, D), 5.0, dtype=BF, device=DEV)
    cuda_lib.qk_norm_rope(q.to(DEV), k.to(DEV), cs.to(DEV), pos.to(DEV), *[None if x is None else x.to(DEV) for x in w],
                          axis_of=axis_of, interleaved=inter, q_out=out[0], k_out=out[1])
    assert cuda_lib.device_status() == (cuda_lib.DEV_BAD_POSITION if bad.any() else 0)
    for x, y, wx in ((q, out[0], w[0]), (k, out[1], w[1])):
        check(y[~bad.to(DEV)], want(x[~bad], wx, cs, pos[:, ~bad], axis_of, inter, 1e-6))
        assert (y[bad.to(DEV)] == 5).all()


def test_rows_by_head_and_a_padded_table(cuda_lib):
    """[heads, T, D] storage on both sides; a table whose rows are not 16-byte aligned."""
    T, H, K, D, R = 19, 6, 2, 64, 64
    g = torch.Generator().manual_seed(5)
    q, k = torch.randn((H, T, D), generator=g).to(BF), torch.randn((K, T, D), generator=g).to(BF)
    cs = table(64, R)
    wide = torch.zeros((64, R + 3))
    wide[:, 1 : R + 1] = cs
    pos = torch.randint(0, 64, (T,), generator=g, dtype=torch.int32)
    qo, ko = torch.empty((H, T, D), dtype=BF, device=DEV), torch.empty((K, T, D), dtype=BF, device=DEV)
    cuda_lib.qk_norm_rope(q.to(DEV).transpose(0, 1), k.to(DEV).transpose(0, 1), wide.to(DEV)[:, 1 : R + 1],
                          pos.to(DEV), q_out=qo.transpose(0, 1), k_out=ko.transpose(0, 1))
    check(qo.transpose(0, 1), want(q.transpose(0, 1), None, cs, pos, None, False, 0))
    check(ko.transpose(0, 1), want(k.transpose(0, 1), None, cs, pos, None, False, 0))


def test_only_one_side_normed_and_special_values(cuda_lib):
    T, D = 4, 64
    q = torch.zeros((T, 1, D), dtype=BF)
    q[0, 0, 3] = float("inf")
    q[1, 0, 5] = float("nan")
    q[2] = 3e38  # the square overflows: the norm gives 0
    k = torch.randn((T, 1, D)).to(BF)
    cs, pos = table(8, D), torch.zeros(T, dtype=torch.int32)
    w = torch.ones(D, dtype=BF)
    qo, ko = cuda_lib.qk_norm_rope(q.to(DEV), k.to(DEV), cs.to(DEV), pos.to(DEV), q_weight=w.to(DEV))
    check(ko, want(k, None, cs, pos, None, False, 0))
    assert torch.isnan(qo[0, 0, 3]) and torch.isnan(qo[1]).all()
    assert (qo[2] == 0).all()
    assert (qo[3] == 0).all()  # zeros: 0 / sqrt(eps)


def test_positions_outside_the_table(cuda_lib):
    T, H, K, D = 40, 3, 2, 128
    g = torch.Generator().manual_seed(3)
    q, k = torch.randn((T, H, D), generator=g).to(BF), torch.randn((T, K, D), generator=g).to(BF)
    cs = table(100, D)
    pos = torch.randint(0, 100, (3, T), generator=g, dtype=torch.int32)
    axis_of = [i // 22 for i in range(64)]
    good = torch.ones(T, dtype=torch.bool)
    for t, a, v in ((0, 0, -1), (7, 2, 100), (39, 1, 2 ** 31 - 1)):
        pos[a, t] = v
        good[t] = False
    qo, ko = torch.full_like(q, 77, device=DEV), torch.full_like(k, 77, device=DEV)
    cuda_lib.qk_norm_rope(q.to(DEV), k.to(DEV), cs.to(DEV), pos.to(DEV), axis_of=axis_of, q_out=qo, k_out=ko)
    assert cuda_lib.device_status() == cuda_lib.DEV_BAD_POSITION
    assert cuda_lib.device_status() == 0
    for got, x in ((qo, q), (ko, k)):
        assert (got[~good.to(DEV)] == 77).all()
        check(got[good.to(DEV)], want(x[good], None, cs, pos[:, good], axis_of, False, 0))


def test_far_positions(cuda_lib):
    """The table's offset passes 32 bits."""
    R, far = 128, 34_000_000
    cs = torch.zeros((far, R), device=DEV)
    pos = torch.tensor([far - 1, 5, 33_600_000], dtype=torch.int32, device=DEV)
    rows = table(3, R).to(DEV)
    cs[pos.long()] = rows
    q = torch.randn((3, 2, R)).to(BF)
    qo, _ = cuda_lib.qk_norm_rope(q.to(DEV), q.to(DEV), cs, pos)
    check(qo, want(q, None, rows.cpu(), torch.arange(3), None, False, 0))


def test_no_tokens(cuda_lib):
    e = torch.empty((0, 2, 64), dtype=BF, device=DEV)
    qo, ko = cuda_lib.qk_norm_rope(e, e, table(4, 64).to(DEV), torch.empty(0, dtype=torch.int32, device=DEV))
    assert qo.shape == e.shape and ko.shape == e.shape


def test_streams_and_graphs(cuda_lib):
    T, H, K, D = 50, 4, 2, 128
    g = torch.Generator().manual_seed(9)
    cs = table(300, D)
    xs = [[torch.randn((T, n, D), generator=g).to(BF) for n in (H, K)] for _ in range(3)]
    ps = [torch.randint(0, 300, (T,), generator=g, dtype=torch.int32) for _ in range(3)]
    ref = [[want(x, None, cs, p, None, False, 0) for x in xx] for xx, p in zip(xs, ps)]
    dcs = cs.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = cuda_lib.qk_norm_rope(xs[0][0].to(DEV), xs[0][1].to(DEV), dcs, ps[0].to(DEV), stream=s)
    q, k, p = xs[1][0].to(DEV), xs[1][1].to(DEV), ps[1].to(DEV)
    here = cuda_lib.qk_norm_rope(q, k, dcs, p)
    torch.cuda.synchronize()
    for got, r in ((side, ref[0]), (here, ref[1])):
        check(got[0], r[0])
        check(got[1], r[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = cuda_lib.qk_norm_rope(q, k, dcs, p)
    q.copy_(xs[2][0]), k.copy_(xs[2][1]), p.copy_(ps[2])
    graph.replay()
    torch.cuda.synchronize()
    check(kept[0], ref[2][0])
    check(kept[1], ref[2][1])
