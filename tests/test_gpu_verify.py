"""Verification of drafted token trees (b2pa_verify_trees) on the GPU, against its definition node by node in 64 bits.

Outputs are whole numbers and have to be equal.  The kernel's values R carry a relative error of about 2^-46 of p
and its sums of V of them 2^-46 of the sum, so that a random number is nearer than that to a border (a tie) with
probability below 2^-46 * 2 V < 2^-28 per token: the inputs here, fixed by their seeds, have none."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BAD_REQUEST, BAD_PROBS = 1, 512


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def sane(row):
    row = row.double()
    return torch.where((row > 0) & (row < float("inf")), row, 0.0)


def reference(target, draft, tokens, parents, uniforms, last, ns):
    """[(path, next token)] of each request: the definition."""
    out, at = [], 0
    for b, n in enumerate(ns):
        if n == 0:
            out.append(([], -1))
            continue
        node, path, V = 0, [0], target.shape[1]
        while True:
            p = sane(target[at + node])
            q = None if draft is None else sane(draft[at + node])
            R, M, a, found = p.clone(), 1.0, 0.0, None
            for i in range(1, n):
                if parents[at + i] != node:
                    continue
                x, u = tokens[at + i], uniforms[at + i]
                r = float(R[x]) if 0 <= x < V else 0.0
                qx = 1.0 if q is None else float(q[x]) if 0 <= x < V else 0.0
                if r > 0 and u * qx * M < r:
                    found = i
                    break
                if q is None:
                    M -= r
                    if 0 <= x < V:
                        R[x] = 0
                elif M > 0:
                    a += M
                    R = (p - a * q).clamp(min=0)
                    M = float(R.sum())
            if found is None:
                break
            node = found
            path.append(node)
        if not float(R.sum()) > 0:
            R = p
        ends = torch.cumsum(R, 0)
        over = (ends > last[b] * float(ends[-1])).nonzero()
        positive = R.nonzero()
        out.append((path, int(over[0]) if len(over) else int(positive[-1]) if len(positive) else -1))
        at += n
    return out


class Trees:
    def __init__(self, ns, V, draft, width=3, seed=0, sharp=3.0, near=1.0, stride=0, offset=0, deep=False):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        T = sum(ns)
        z = torch.randn((T, V), generator=g) * sharp
        self.ns, self.V = ns, V

        def rows(x):
            if not stride:
                return x
            wide = torch.full((T, stride), float("nan"))
            wide[:, offset : offset + V] = x
            return wide[:, offset : offset + V]

        self.target = rows(torch.softmax(z + near * torch.randn((T, V), generator=g), -1))
        self.draft = rows(torch.softmax(z, -1)) if draft else None
        self.parents, self.tokens, at = [], [], 0
        for n in ns:
            kids = [0] * n
            for i in range(n):
                up = -1
                if i:
                    up = i - 1 if deep else r.choice([j for j in range(i) if kids[j] < width])
                    kids[up] += 1
                self.parents.append(up if i else 12345)  # the root's is not read
                if not i:
                    self.tokens.append(-7)
                elif draft:
                    self.tokens.append(int(torch.multinomial(self.draft[at + up], 1, generator=g)))
                else:  # the draft's likeliest, or, where there is no other, one of them again
                    best = torch.topk(z[at + up], min(V, width)).indices
                    self.tokens.append(int(best[(kids[up] - 1) % len(best)]))
            at += n
        self.uniforms = torch.rand(T, generator=g)
        self.last = torch.rand(len(ns), generator=g)

    def args(self):
        d = lambda x: None if x is None else x.to(DEV) if x.is_contiguous() else wide(x)  # noqa: E731

        def wide(x):  # the same strides and offset on the GPU
            base = x._base.to(DEV)
            return base.as_strided(x.shape, x.stride(), x.storage_offset())

        return dict(target_probs=d(self.target), tokens=ints(self.tokens), parents=ints(self.parents),
                    uniforms=d(self.uniforms), last_uniforms=d(self.last), max_q_len=max(self.ns + [0]),
                    cum_seq_lens_q=ints([sum(self.ns[:i]) for i in range(len(self.ns) + 1)]), draft_probs=d(self.draft))

    def want(self):
        return reference(self.target, self.draft, self.tokens, self.parents, self.uniforms.tolist(), self.last.tolist(),
                         self.ns)

    def check(self, got, width=None):
        acc, cnt, nxt = (x.tolist() for x in got)
        lengths = []
        for b, (path, token) in enumerate(self.want()):
            assert (cnt[b], nxt[b]) == (len(path), token), (b, path, token, acc[b])
            assert acc[b] == path + [-1] * ((width or max(self.ns + [0])) - len(path)), b
            lengths.append(len(path))
        return lengths


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [1, 2, 5, 127, 128, 129, 1000, 2048, 2049, 32000, 50257, 131072])
def test_vocabularies(cuda_lib, draft, V):
    """Every size where a run of values ends; several trees, one of no nodes and one of the root alone."""
    x = Trees([5, 1, 0, 9, 14], V, draft, seed=V + draft)
    x.check(cuda_lib.verify_trees(**x.args()))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("stride,offset", [(1037, 0), (1036, 4), (1040, 3), (1041, 17)])
def test_rows_that_are_not_aligned(cuda_lib, draft, stride, offset):
    x = Trees([7, 20, 3], 1003, draft, seed=stride, stride=stride, offset=offset)
    x.check(cuda_lib.verify_trees(**x.args()))


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("near,sharp", [(0.0, 2.0), (0.3, 3.0), (4.0, 6.0)])
def test_batches(cuda_lib, draft, near, sharp):
    """Paths long and short: drafts equal to the target, near it and far from it; chains and wide trees."""
    r = random.Random(1)
    x = Trees([r.randint(1, 30) for _ in range(120)], 300, draft, 4, seed=5, sharp=sharp, near=near)
    some = x.check(cuda_lib.verify_trees(**x.args()))
    y = Trees([r.randint(1, 64) for _ in range(40)], 300, draft, 1, seed=6, sharp=sharp, near=near, deep=True)
    some += y.check(cuda_lib.verify_trees(**y.args()))
    assert max(some) > 2 or near > 1
    assert cuda_lib.device_status() == 0


def test_equal_draft_is_always_accepted(cuda_lib):
    """p = q: u q < p for every u < 1, down to the chain's end."""
    x = Trees([40, 64, 2], 5000, True, 1, seed=3, near=0.0, deep=True)
    x.draft = x.target.clone()
    x.uniforms.fill_(1 - 2.0 ** -24)
    got = cuda_lib.verify_trees(**x.args())
    x.check(got)
    assert got[1].tolist() == [40, 64, 2]


@pytest.mark.parametrize("draft", [False, True])
def test_a_wide_tree(cuda_lib, draft):
    """4096 nodes: many children, many refusals, and the most that a call may have."""
    for n, width in ((4096, 200), (300, 299), (1000, 31)):
        x = Trees([n, 5], 700, draft, width, seed=n, near=3.0)
        x.uniforms.mul_(0.5).add_(0.5)
        x.check(cuda_lib.verify_trees(**x.args()))
    assert cuda_lib.device_status() == 0


def test_twins(cuda_lib):
    """The same token drafted twice by one node: refused once, it has nothing left."""
    x = Trees([6], 10, False, 5, seed=1)
    x.parents, x.tokens = [-1, 0, 0, 0, 0, 0], [0, 4, 4, 7, 4, 7]
    x.target[0] = torch.tensor([0, 0, 0, 0, 0.5, 0, 0, 0.25, 0.125, 0.125])
    for u, path, token in (((0.6, 0.0, 0.6, 0.0, 0.0), [0], 8), ((0.6, 0.0, 0.4, 0.0, 0.0), [0, 3], None),
                           ((0.4, 0.9, 0.9, 0.9, 0.9), [0, 1], None), ((0.5, 0.5, 0.5, 0.5, 0.5), [0], 8)):
        x.uniforms = torch.tensor([0.0, *u])
        x.last = torch.tensor([0.25])
        got = cuda_lib.verify_trees(**x.args())
        x.check(got)
        assert got[0].tolist()[0][: len(path)] == path and token in (None, int(got[2]))


@pytest.mark.parametrize("draft", [False, True])
def test_nothing_left(cuda_lib, draft):
    """All of p refused: the next token comes from p itself.  (0.75 >= p(x) = 1 never: u at its end, q larger.)"""
    V = 2000
    x = Trees([3, 3], V, draft, 2, seed=1)
    x.parents, x.tokens = [-1, 0, 0, -1, 0, 0], [0, 9, 9, 0, 5, 6]
    x.target.zero_()
    x.target[:, 9] = 0.5  # rows of sum 0.5: refused at u = 0.75
    x.target[3:, 9], x.target[3:, 5], x.target[3:, 6] = 0, 0.25, 0.25
    if draft:
        x.draft = x.target * 2
    x.uniforms.fill_(0.75)
    for v in (0.0, 0.3, 0.75, 1 - 2.0 ** -24):
        x.last.fill_(v)
        got = cuda_lib.verify_trees(**x.args())
        x.check(got)
        assert int(got[2][0]) == 9
    assert cuda_lib.device_status() == 0


def test_values_that_are_not_probabilities(cuda_lib):
    """NaN, infinities and values below 0 count as 0; tokens outside the vocabulary are refused."""
    for draft in (False, True):
        x = Trees([12, 12, 4], 600, draft, 3, seed=2)
        for t in (x.target, x.draft):
            if t is not None:
                for k, v in enumerate((float("nan"), float("inf"), -float("inf"), -0.25)):
                    t[:, k::37] = v
        x.tokens[3], x.tokens[5], x.tokens[14] = -1, 600, 2 ** 31 - 1
        x.uniforms[7] = float("nan")
        x.check(cuda_lib.verify_trees(**x.args()))
        assert cuda_lib.device_status() == 0
        x.target[:12] = float("nan")
        x.target[24:] = 0
        got = cuda_lib.verify_trees(**x.args())
        x.check(got)
        assert got[2].tolist()[0] == -1 and got[1].tolist()[0] == 1
        assert cuda_lib.device_status() == BAD_PROBS


def test_last_numbers_at_their_ends(cuda_lib):
    """0 takes the first positive value, and 1 (not allowed), or what rounds to it, the last."""
    x = Trees([1] * 4, 1500, False, seed=4)
    x.target[:, :300] = 0
    x.target[:, 1200:] = 0
    x.last = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 2.0])
    got = cuda_lib.verify_trees(**x.args())
    x.check(got)
    assert got[2].tolist()[0] == 300 and got[2].tolist()[2:] == [1199, 1199]


def test_small_and_large_values_together(cuda_lib):
    """A tail of values 2^-40 of the largest: a sum in 32 bits loses it, the draw behind it must not."""
    V = 65536
    x = Trees([1, 1, 1], V, False, seed=8)
    x.target[:] = 2.0 ** -40
    x.target[:, 77] = 1.0
    x.last = torch.tensor([1 - 2.0 ** -24, 2.0 ** -37, 2.0 ** -36])
    x.check(cuda_lib.verify_trees(**x.args()))


def test_malformed_requests(cuda_lib):
    """Parents behind their children, trees beyond max_q_len, rows outside the batch: count 0, token -1, and the
    others as if they were alone."""
    x = Trees([5, 6, 4, 7, 5], 200, True, 2, seed=9)
    good = cuda_lib.verify_trees(**x.args())
    a = x.args()
    a["parents"][5 + 3] = 3   # itself
    a["parents"][11 + 2] = -1
    a["max_q_len"] = 6        # less than request 3's seven
    a["cum_seq_lens_q"][5] = 28
    acc, cnt, nxt = cuda_lib.verify_trees(**a)
    assert cnt.tolist() == [good[1].tolist()[0], 0, 0, 0, 0] and nxt.tolist() == [good[2].tolist()[0], -1, -1, -1, -1]
    assert acc[0].tolist() == good[0][0, :6].tolist() and bool((acc[1:] == -1).all())
    assert cuda_lib.device_status() == BAD_REQUEST


def test_outputs_given(cuda_lib):
    """Wider rows with a stride; an empty batch."""
    x = Trees([9, 3], 400, False, seed=2)
    wide = torch.full((2, 20), 5, dtype=torch.int32, device=DEV)
    cnt, nxt = ints([7, 7]), ints([7, 7])
    got = cuda_lib.verify_trees(**x.args(), accepted=wide[:, :13], num_accepted=cnt, next_tokens=nxt)
    assert got[1] is cnt and got[2] is nxt and bool((wide[:, 13:] == 5).all())
    x.check(got, 13)
    e = torch.empty(0, device=DEV)
    got = cuda_lib.verify_trees(torch.empty((0, 50), device=DEV), e.int(), e.int(), e, e, 4, ints([0]))
    assert [list(t.shape) for t in got] == [[0, 4], [0], [0]]


@pytest.mark.parametrize("draft", [False, True])
def test_tokens_are_distributed_as_the_target(cuda_lib, draft):
    """The first token that comes out of N requests has the target's distribution, whatever the draft.  A count of N
    draws with probability p is off its mean by less than 5 sqrt(N p (1 - p)) but for once in 1.7 million."""
    N, V = 60000, 12
    g = torch.Generator(device=DEV).manual_seed(11 + draft)
    p = torch.softmax(torch.randn(V, generator=g, device=DEV) * 1.5, 0)
    q = torch.softmax(torch.randn(V, generator=g, device=DEV) * 1.5, 0)
    n = 4  # the root and three children
    target = p.expand(N * n, V).contiguous()
    parents = ints([-1, 0, 0, 0]).repeat(N)
    if draft:
        tokens = torch.multinomial(q.expand(N, V), n, replacement=True, generator=g).int().view(-1)
    else:
        tokens = torch.topk(q, n).indices.int().repeat(N)
    u = torch.rand(N * n, generator=g, device=DEV)
    acc, cnt, nxt = cuda_lib.verify_trees(target, tokens, parents, u, torch.rand(N, generator=g, device=DEV), n,
                                          torch.arange(N + 1, device=DEV, dtype=torch.int32) * n,
                                          draft_probs=q.expand(N * n, V).contiguous() if draft else None)
    first = torch.where(cnt > 1, tokens.view(N, n).gather(1, acc[:, 1:2].clamp(min=0).long())[:, 0], nxt)
    seen = torch.bincount(first.long(), minlength=V).double()
    p = p.double()
    assert bool(((seen - N * p).abs() <= 5 * torch.sqrt(N * p * (1 - p))).all())


def test_rows_behind_32_bits(cuda_lib):
    """Rows whose elements lie past 2^31."""
    V, n = 262144, 8200
    target = torch.zeros((n, V), device=DEV)
    target[:, 5] = 1.0
    target[n - 2, 5], target[n - 2, 99] = 0, 1.0
    target[n - 1, 5], target[n - 1, V - 1] = 0, 1.0
    cum = ints([0, n - 2, n])
    parents = torch.zeros(n, dtype=torch.int32, device=DEV)
    tokens = ints([99] * n)
    half = torch.full((n,), 0.5, device=DEV)
    acc, cnt, nxt = cuda_lib.verify_trees(target, tokens, parents, half, half[:2], 4, cum)
    assert cnt.tolist() == [0, 2] and nxt.tolist() == [-1, V - 1]  # (the first has more nodes than it may)
    assert cuda_lib.device_status() == BAD_REQUEST


def test_streams_and_graphs(cuda_lib):
    """A call on a named stream, behind what waits there; two captured calls at once, replayed on new inputs."""
    x, y = Trees([9, 14, 3], 3000, True, seed=1), Trees([9, 14, 3], 3000, True, seed=2)
    a, b = x.args(), y.args()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    cuda_lib.verify_trees(**a, stream=side)
    torch.cuda.synchronize()
    inputs = {k: v.clone() for k, v in a.items() if isinstance(v, torch.Tensor)}
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for k, v in inputs.items():
            v.copy_(b[k])
    call = {**a, **inputs}
    got = cuda_lib.verify_trees(**call, stream=side)
    side.synchronize()
    y.check(got)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph, stream=side):
            outs.append(cuda_lib.verify_trees(**call))
    for want, args in ((x, a), (y, b)):
        for k, v in inputs.items():
            v.copy_(args[k])
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        want.check(outs[0])
        want.check(outs[1])
