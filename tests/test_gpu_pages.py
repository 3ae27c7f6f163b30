"""The page ledger, page copies and the compaction of accepted nodes on the GPU, against the same steps one by one
in Python.  Nothing is computed: every comparison is of bits."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
BAD_REQUEST, BAD_PAGE, NO_PAGES = 1, 2, 256


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- ledger

class Ledger:
    """The definition: lists, and the device's tensors beside them."""

    def __init__(self, R, N, P, width, seed=0, stride=None):
        r = random.Random(seed)
        self.P, self.N, self.R = P, N, R
        self.table = [[r.randrange(-5, N + 5) for _ in range(width)] for _ in range(R)]  # leftovers of other requests
        self.seq, self.refs = [0] * R, [0] * N
        self.stride = stride or width
        self.width = width
        self.r = r

    def fill(self, row, tokens, pages=None):
        n = -(-tokens // self.P)
        free = [i for i in range(self.N) if self.refs[i] == 0]
        pages = pages or self.r.sample(free, n)
        for c, pg in enumerate(pages):
            self.table[row][c] = pg
            self.refs[pg] += 1
        self.seq[row] = tokens

    def dev(self):
        self.t = torch.zeros((self.R, self.stride), dtype=torch.int32, device=DEV)[:, : self.width]
        self.t.copy_(torch.tensor(self.table, dtype=torch.int32))
        self.s, self.c = ints(self.seq), ints(self.refs)
        return self

    def same(self):
        assert self.t.tolist() == self.table
        assert self.s.tolist() == self.seq
        assert self.c.tolist() == self.refs

    def pages(self, tokens):
        return -(-tokens // self.P)

    def free(self, rows):
        for r in rows:
            for pg in self.table[r][: self.pages(self.seq[r])]:
                self.refs[pg] -= 1
            self.seq[r] = 0

    def take(self, wants):
        """Pages of each request: the lowest free ones in order, all or none."""
        free, at, out = [i for i, x in enumerate(self.refs) if x == 0], 0, []
        for w in wants:
            out.append(free[at : at + w] if at + w <= len(free) else None)
            at += w
        return out

    def fork(self, parents, children):
        src, dst, bad = [], [], 0
        ok, seen = [], set()
        for p, c in zip(parents, children):
            good = 0 <= c < self.R and 0 <= p < self.R and c not in seen and c not in parents
            good = good and self.seq[c] == 0 and 0 <= self.pages(self.seq[p]) <= self.width
            if 0 <= c < self.R:
                seen.add(c)
            ok.append(good)
            bad |= 0 if good else BAD_REQUEST
        got = self.take([int(g and self.seq[p] % self.P != 0) for g, p in zip(ok, parents)])
        for g, p, c, pg in zip(ok, parents, children, got):
            src.append(-1)
            dst.append(-1)
            if not g:
                continue
            if pg is None and self.seq[p] % self.P:
                bad |= NO_PAGES
                continue
            whole = self.seq[p] // self.P
            for i in range(whole):
                self.table[c][i] = self.table[p][i]
                self.refs[self.table[p][i]] += 1
            if self.seq[p] % self.P:
                src[-1], dst[-1] = self.table[p][whole], pg[0]
                self.table[c][whole] = pg[0]
                self.refs[pg[0]] = 1
            self.seq[c] = self.seq[p]
        return src, dst, bad

    def grow(self, rows, to):
        bad, ok, seen, back = 0, [], set(), []
        for r, t in zip(rows, to):
            good = 0 <= r < self.R and r not in seen and t >= 0 and self.pages(t) <= self.width
            if 0 <= r < self.R:
                seen.add(r)
            ok.append(good)
            bad |= 0 if good else BAD_REQUEST
        wants = [max(self.pages(t) - self.pages(self.seq[r]), 0) if g else 0 for g, r, t in zip(ok, rows, to)]
        for g, r, t, w, got in zip(ok, rows, to, wants, self.take(wants)):
            if not g:
                continue
            if w and got is None:
                bad |= NO_PAGES
                continue
            first = self.pages(self.seq[r])
            for i in range(w):
                self.table[r][first + i] = got[i]
                self.refs[got[i]] = 1
            back += self.table[r][self.pages(t) : first]
            self.seq[r] = t
        for pg in back:  # free from the next call on
            self.refs[pg] -= 1
        return bad


def run_fork(b2pa, led, parents, children):
    src, dst, bad = led.fork(parents, children)
    got = b2pa.fork_pages(led.t, led.s, led.c, ints(parents), ints(children), led.P)
    assert got[0].tolist() == src and got[1].tolist() == dst
    led.same()
    assert b2pa.device_status() == bad


def run_grow(b2pa, led, rows, to):
    bad = led.grow(rows, to)
    b2pa.grow_pages(led.t, led.s, led.c, ints(rows), ints(to), led.P)
    led.same()
    assert b2pa.device_status() == bad


def run_free(b2pa, led, rows, call=None):
    led.free(rows)
    b2pa.free_pages(led.t, led.s, led.c, ints(call or rows), led.P)
    led.same()
    assert b2pa.device_status() == 0


@pytest.mark.parametrize("P", [1, 16, 48])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_ledger_of_random_steps(cuda_lib, P, seed):
    """Rows come, grow, fork and go, until pages run out and come back."""
    r = random.Random(seed)
    led = Ledger(40, 301, P, 33, seed, stride=37).dev()
    for step in range(25):
        empty = [i for i in range(led.R) if led.seq[i] == 0]
        full = [i for i in range(led.R) if led.seq[i]]
        what = r.choice(["grow", "fork", "free", "grow"])
        if what == "grow":
            rows = r.sample(range(led.R), r.randint(1, 12))
            run_grow(cuda_lib, led, rows, [max(0, min(33 * P, led.seq[i] + r.choice([0, 1, P, -1, r.randint(-9 * P, 9 * P)])))
                                           for i in rows])
        elif what == "fork" and full and empty:
            kids = r.sample(empty, r.randint(1, len(empty)))
            run_fork(cuda_lib, led, [r.choice(full) for _ in kids], kids)
        elif what == "free" and full:
            run_free(cuda_lib, led, r.sample(full, r.randint(1, len(full))))


@pytest.mark.parametrize("N", [1, 31, 1023, 1024, 1025, 4099, 70001])
def test_lowest_free_pages(cuda_lib, N):
    """The free pages anywhere, the last one among them, and none left at the end."""
    led = Ledger(3, N, 4, N + 1, N)
    led.refs = [led.r.choice([1, 1, 2]) for _ in range(N)]
    for i in led.r.sample(range(N), max(1, N // 50)) + [N - 1]:
        led.refs[i] = 0
    led.dev()
    free = led.refs.count(0)
    run_grow(cuda_lib, led, [2], [4 * (free - 1)])
    run_grow(cuda_lib, led, [0, 1], [4, 5])
    run_grow(cuda_lib, led, [1, 0], [5, 3])


def test_many_requests(cuda_lib):
    """As many as a call may have."""
    R = 4096
    led = Ledger(2 * R, 5 * R, 8, 6, 5)
    order = led.r.sample(range(5 * R), 5 * R)
    at = 0
    for i in range(R):
        n = led.r.randint(0, 24)
        led.fill(i, n, order[at : at + led.pages(n)])
        at += led.pages(n)
    led.dev()
    run_fork(cuda_lib, led, [led.r.randrange(R) for _ in range(R)], led.r.sample(range(R, 2 * R), R))
    run_grow(cuda_lib, led, list(range(R)), [led.seq[i] + led.r.randint(0, 16) for i in range(R)])
    run_free(cuda_lib, led, list(range(R, 2 * R)))


def test_fork_of_parents_on_page_borders(cuda_lib):
    """Lengths of 0, a page, one more and one less; a parent with many children; leftovers behind the length stay."""
    led = Ledger(20, 50, 16, 5, 7)
    for row, n in enumerate([0, 16, 17, 15, 1, 80]):
        led.fill(row, n)
    led.dev()
    run_fork(cuda_lib, led, [0, 1, 2, 3, 4, 5, 2, 2, 5], [10, 11, 12, 13, 14, 15, 16, 17, 18])


@pytest.mark.parametrize("bad", [-1, -3, 40, 2 ** 31 - 1])
def test_fork_of_a_last_page_outside_the_pool(cuda_lib, bad):
    """Flagged; the child has a page of its own there, and what there is to copy names the page as it stands, so that
    the copy passes it over and flags it too.  Pages of parents that are whole are flagged as before."""
    led = Ledger(5, 40, 16, 4)
    led.fill(0, 50)
    led.fill(1, 39)
    led.table[0][3] = bad
    led.dev()
    src, dst = cuda_lib.fork_pages(led.t, led.s, led.c, ints([0, 1]), ints([2, 3]), 16)
    assert cuda_lib.device_status() == BAD_PAGE
    free = [i for i in range(40) if led.refs[i] == 0]
    assert src.tolist() == [bad, led.table[1][2]] and dst.tolist() == free[:2]
    assert led.s.tolist() == [50, 39, 50, 39, 0]
    assert led.t[2].tolist() == led.table[0][:3] + [free[0]] and led.t[3, :3].tolist() == led.table[1][:2] + [free[1]]
    pool = torch.randint(0, 100, (40, 2, 16, 16), device=DEV).to(torch.bfloat16)
    k, v = pool.clone(), pool.clone()
    cuda_lib.copy_pages((k, v), src, dst)
    assert cuda_lib.device_status() == BAD_PAGE
    pool[free[1]] = pool[led.table[1][2]]
    assert torch.equal(k, pool) and torch.equal(v, pool)


def test_requests_that_are_malformed(cuda_lib):
    """They change nothing, and those beside them are served."""
    led = Ledger(12, 60, 16, 4, 9)
    for row, n in enumerate([20, 30, 64, 5]):
        led.fill(row, n)
    led.dev()
    # rows outside the table, a child twice, one that is a parent, one that is not empty
    run_fork(cuda_lib, led, [0, -1, 12, 0, 1, 4, 0, 2], [4, 5, 6, 4, 12, 7, 3, 8])
    run_grow(cuda_lib, led, [0, 0, 1, 2, -3, 9, 3], [25, 40, 29, 65, 5, 64, -1])


def test_pages_run_out(cuda_lib):
    """A request short of pages stays as it was; those before it are served, later ones with enough left are not by chance."""
    led = Ledger(12, 12, 4, 8, 3)
    led.fill(0, 18)
    led.fill(1, 2)
    led.dev()
    run_grow(cuda_lib, led, [2, 3, 4, 5], [8, 32, 0, 4])   # 2 of 6 free, 8 wanted, none wanted, then 1
    run_fork(cuda_lib, led, [0, 1, 0, 1, 0, 1], [6, 7, 8, 9, 10, 11])
    run_grow(cuda_lib, led, [2], [12])


def test_more_pages_wanted_than_an_int_counts(cuda_lib):
    """Sums of what requests want end at their limit instead of wrapping."""
    most = (1 << 30) - 1
    table = torch.empty((5, most), dtype=torch.int32, device=DEV)  # 20 GB that nothing reads
    table[3, :2] = -1
    seq, refs = ints([0] * 5), ints([1, 0, 0, 1])
    cuda_lib.grow_pages(table, seq, refs, ints([3, 0, 1, 2, 4]), ints([1, most, most, most, 1]), 1)
    assert seq.tolist() == [0, 0, 0, 1, 0] and refs.tolist() == [1, 1, 0, 1] and table[3, :2].tolist() == [1, -1]
    assert cuda_lib.device_status() == NO_PAGES


def test_arguments_between_the_rows_of_a_table(cuda_lib):
    """The room behind a table's rows is no part of it: lengths and rows may lie there."""
    led = Ledger(6, 40, 16, 4, 3, stride=12)
    led.fill(0, 20)
    led.dev()
    room = led.t.as_strided((6, 12), (12, 1))
    room[2, 4:7], room[3, 4:7] = ints([0, 1, 3]), ints([33, 16, 1])
    bad = led.grow([0, 1, 3], [33, 16, 1])
    cuda_lib.grow_pages(led.t, led.s, led.c, room[2, 4:7], room[3, 4:7], 16)
    led.same()
    assert cuda_lib.device_status() == bad == 0
    src, dst, bad = led.fork([0, 1], [2, 4])
    cuda_lib.fork_pages(led.t, led.s, led.c, ints([0, 1]), ints([2, 4]), 16, src=room[5, 5:7], dst=room[5, 7:9])
    led.same()
    assert room[5, 5:9].tolist() == src + dst and cuda_lib.device_status() == bad == 0
    assert room[2, 4:7].tolist() == [0, 1, 3] and (room[0, 4:] == 0).all()


def test_rows_that_become_shorter(cuda_lib):
    """Pages behind the new length go back, those that others hold stay theirs, and nobody gets them in the same call."""
    led = Ledger(8, 12, 4, 9, 4)
    led.fill(0, 33)
    led.dev()
    run_grow(cuda_lib, led, [0, 1, 2], [5, 12, 1])   # 3 free pages: the first two thirds of what is asked for
    run_grow(cuda_lib, led, [2, 1, 0], [4, 36, 0])
    run_fork(cuda_lib, led, [1], [3])
    run_grow(cuda_lib, led, [1, 3], [1, 40])
    run_grow(cuda_lib, led, [3], [0])


def test_free_twice(cuda_lib):
    """A row named twice is freed once; pages of two rows that fall together; counts of 0 stay."""
    led = Ledger(6, 30, 8, 4, 2)
    led.fill(0, 30)
    led.fill(1, 30, led.table[0][:4])
    led.fill(2, 9)
    led.dev()
    run_free(cuda_lib, led, [0, 1, 2, 5], [0, 1, 0, 2, 1, 5])
    led.fill(3, 20)
    led.refs[led.table[3][1]] = 0
    led.dev()
    cuda_lib.free_pages(led.t, led.s, led.c, ints([3, 6, -1]), 8)
    assert cuda_lib.device_status() == BAD_PAGE | BAD_REQUEST
    led.refs = [0] * 30
    led.seq[3] = 0
    led.same()


# ---------------------------------------------------------------- pools

def make_pools(N, Hkv, P, D, layout, cache, seed, strided=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (N, Hkv, P, D) if layout == "HND" else (N, P, Hkv, D)

    def one():
        if strided:  # the two halves of one [N, 2, ...] tensor, in wider rows
            full = torch.randint(0, 256, (N, 2, *shape[1:-1], D + 8), generator=g, device=DEV, dtype=torch.uint8)
            return full[:, 1, :, :, :D]
        return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)

    if cache == "bf16":
        def make():
            wide = torch.randint(-2 ** 15, 2 ** 15, (*shape[:-1], D + (8 if strided else 0)), generator=g, device=DEV,
                                 dtype=torch.int16)
            return wide[..., :D].view(torch.bfloat16)
        pools = (make(), make())
    else:
        pools = (one().view(F8), one().view(F8))
    scales = None
    if cache == "scaled":
        scales = tuple(torch.randn((*shape[:-1], 2), generator=g, device=DEV)[..., 0] if strided
                       else torch.randn(shape[:-1], generator=g, device=DEV) for _ in "kv")
    return pools, scales


def bits(x):
    return x.view(torch.int16) if x.dtype == torch.bfloat16 else x.view(torch.uint8) if x.dtype == F8 else x


POOLS = [
    # N, Hkv, P, D, layout, cache, strided
    (9, 8, 32, 128, "HND", "bf16", False),
    (9, 8, 64, 128, "NHD", "scaled", False),
    (7, 2, 16, 64, "HND", "e4m3", True),
    (7, 3, 5, 80, "NHD", "scaled", True),
    (5, 1, 1, 8, "HND", "scaled", False),
    (6, 5, 3, 7, "NHD", "bf16", False),     # rows of 14 bytes
    (6, 2, 4, 33, "HND", "e4m3", False),    # rows of 33 bytes
    (5, 1, 128, 256, "HND", "bf16", True),
]


@pytest.mark.parametrize("N,Hkv,P,D,layout,cache,strided", POOLS)
def test_copy_pages(cuda_lib, N, Hkv, P, D, layout, cache, strided):
    pools, scales = make_pools(N, Hkv, P, D, layout, cache, 1, strided)
    planes = [*pools, *(scales or ())]
    want = [bits(x).clone() for x in planes]
    src, dst = [0, -1, 0, 1], [N - 1, -1, 2, 3]
    for x in want:
        for a, b in zip(src, dst):
            if a >= 0:
                x[b] = x[a]
    cuda_lib.copy_pages(pools, ints(src), ints(dst), kv_scales=scales, kv_layout=layout)
    for x, y in zip(planes, want):
        assert torch.equal(bits(x), y)
    # pages that are none are passed over, and the pairs beside them are not
    for x in want:
        x[1] = x[0]
    cuda_lib.copy_pages(pools, ints([N, 0, -1, 2]), ints([0, 1, 0, -2]), kv_scales=scales, kv_layout=layout)
    assert cuda_lib.device_status() == BAD_PAGE
    for x, y in zip(planes, want):
        assert torch.equal(bits(x), y)
    cuda_lib.copy_pages(pools, ints([]), ints([]), kv_scales=scales, kv_layout=layout)


def test_copy_pages_behind_32_bits(cuda_lib):
    """Pages whose elements lie past 2^31."""
    N = 40000
    pools = tuple(torch.zeros((N, 8, 64, 128), dtype=F8, device=DEV) for _ in "kv")  # 65536 bytes a page
    for x in pools:
        bits(x)[N - 2] = torch.randint(0, 256, (8, 64, 128), device=DEV, dtype=torch.uint8)
    cuda_lib.copy_pages(pools, ints([N - 2, 0]), ints([N - 1, N - 3]))
    for x in pools:
        assert torch.equal(bits(x)[N - 1], bits(x)[N - 2]) and int(bits(x)[N - 3].sum()) == 0
    assert cuda_lib.device_status() == 0


def compact_by_hand(planes, layout, table, kvs, ns, accepted, P):
    for x in planes:
        y = x.transpose(1, 2) if layout == "HND" else x
        for b, path in enumerate(accepted):
            c = kvs[b] - ns[b]
            rows = [y[table[b][(c + a) // P], (c + a) % P].clone() for a in path]
            for i, row in enumerate(rows):
                y[table[b][(c + i) // P], (c + i) % P] = row


@pytest.mark.parametrize("N,Hkv,P,D,layout,cache,strided", POOLS)
@pytest.mark.parametrize("seed", [1, 2])
def test_compact(cuda_lib, N, Hkv, P, D, layout, cache, strided, seed):
    """Paths whose places overlap the nodes that follow, over page borders; nothing taken, all taken, no tree."""
    r = random.Random(seed)
    ns = [7, 1, 0, 40, 12, 33, 9]
    kvs = [n + r.randint(0, 3 * P) for n in ns]
    used = [-(-k // P) for k in kvs]
    N = sum(used) + 2
    pools, scales = make_pools(N, Hkv, P, D, layout, cache, seed, strided)
    order = r.sample(range(N), N)
    table = [[order.pop() for _ in range(u)] + [-9] * (max(used) + 1 - u) for u in used]
    counts = [r.randint(0, n) for n in ns]
    counts[0], counts[3] = 7, r.randint(20, 39)
    accepted = [sorted(r.sample(range(n), k)) for n, k in zip(ns, counts)]
    accepted[5], accepted[6] = list(range(1, 33)), [8]  # everything one place down; the last node alone
    counts[5], counts[6] = 32, 1
    planes = [*pools, *(scales or ())]
    want = [bits(x).clone() for x in planes]
    compact_by_hand(want, layout, table, kvs, ns, accepted, P)
    acc = torch.full((len(ns), 45), 12345, dtype=torch.int32)
    for b, path in enumerate(accepted):
        acc[b, : len(path)] = torch.tensor(path, dtype=torch.int32)
    lens = cuda_lib.compact_kv(pools, ints(table), ints(kvs), ints([sum(ns[:i]) for i in range(8)]),
                               acc.to(DEV)[:, :41], ints(counts), kv_scales=scales, kv_layout=layout)
    assert lens.tolist() == [k - n + c for k, n, c in zip(kvs, ns, counts)]
    for x, y in zip(planes, want):
        assert torch.equal(bits(x), y)
    assert cuda_lib.device_status() == 0


def test_compact_of_malformed_requests(cuda_lib):
    """Nodes that do not rise, that are none, counts that cannot be, trees longer than their requests: nothing
    moves; a page that is none: its rows stay."""
    P, ns, kvs = 4, [4, 4, 4, 4, 9, 4, 4], [8, 8, 8, 8, 8, 8, 100]
    pools, _ = make_pools(16, 2, P, 16, "HND", "bf16", 3)
    want = [bits(x).clone() for x in pools]
    table = [[2 * b, 2 * b + 1] for b in range(7)]
    accepted = [[1, 1, 0], [0, 4, 0], [2, 3, 0], [-1, 0, 0], [1, 2, 3], [1, 3, 0], [0, 1, 2]]
    counts = [2, 2, 5, 2, 3, 2, 2]
    table[5][1] = 77
    out = torch.full((7,), -5, dtype=torch.int32, device=DEV)
    lens = cuda_lib.compact_kv(pools, ints(table), ints(kvs), ints([0, 4, 8, 12, 16, 25, 29, 33]), ints(accepted),
                               ints(counts), new_lens=out)
    assert lens is out and lens.tolist() == [8, 8, 8, 8, 8, 6, 100]
    for x, y in zip(pools, want):
        assert torch.equal(bits(x), y)
    assert cuda_lib.device_status() == BAD_REQUEST | BAD_PAGE


# ---------------------------------------------------------------- streams and graphs

def test_a_captured_step(cuda_lib):
    """free, fork, grow and copy in one graph, replayed: the same step again each time."""
    led = Ledger(12, 200, 16, 20, 4)
    led.fill(0, 100)
    led.fill(1, 77)
    for row in range(2, 8):
        led.fill(row, led.r.randint(1, 150))
    led.dev()
    pools, _ = make_pools(200, 2, 16, 64, "HND", "bf16", 5)
    kids, parents, to = list(range(2, 8)), [0, 0, 1, 1, 0, 1], [130, 100, 90, 77, 200, 120]
    dk, dp, dt = ints(kids), ints(parents), ints(to)

    def step():
        cuda_lib.free_pages(led.t, led.s, led.c, dk, 16)
        src, dst = cuda_lib.fork_pages(led.t, led.s, led.c, dp, dk, 16)
        cuda_lib.grow_pages(led.t, led.s, led.c, dk, dt, 16)
        cuda_lib.copy_pages(pools, src, dst)
        return src, dst

    cuda_lib.free_pages(led.t, led.s, led.c, ints([]), 16)
    cuda_lib.device_status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the first call on a stream is not captured
        cuda_lib.copy_pages(pools, ints([-1]), ints([-1]))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        src, dst = step()
    led.same()  # (nothing has run)
    want = [bits(x).clone() for x in pools]
    for _ in range(3):
        led.free(kids)
        s, d, bad = led.fork(parents, kids)
        assert bad == 0 and led.grow(kids, to) == 0
        for x in want:
            for a, b in zip(s, d):
                if a >= 0:
                    x[b] = x[a]
        graph.replay()
        torch.cuda.synchronize()
        led.same()
        assert src.tolist() == s and dst.tolist() == d
        for x, y in zip(pools, want):
            assert torch.equal(bits(x), y)
    assert cuda_lib.device_status(side) == 0


def test_calls_on_a_named_stream(cuda_lib):
    """Every call runs on the stream it names, behind what waits there."""
    side = torch.cuda.Stream()
    led = Ledger(6, 40, 8, 6, 1)
    led.fill(0, 21)
    led.dev()
    pools, _ = make_pools(40, 2, 8, 64, "HND", "bf16", 6)
    torch.cuda.synchronize()
    rows, kids, to = ints([0, 0]), ints([1, 2]), ints([30, 40])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late = bits(pools[0])
        late[led.table[0][2]] = 7
    src, dst = cuda_lib.fork_pages(led.t, led.s, led.c, rows, kids, 8, stream=side)
    cuda_lib.grow_pages(led.t, led.s, led.c, kids, to, 8, stream=side)
    cuda_lib.copy_pages(pools, src, dst, stream=side)
    cuda_lib.free_pages(led.t, led.s, led.c, kids[:1], 8, stream=side)
    side.synchronize()
    s, d, _ = led.fork([0, 0], [1, 2])
    led.grow([1, 2], [30, 40])
    led.free([1])
    led.same()
    for page in d:
        assert int((bits(pools[0])[page] != 7).sum()) == 0
    assert cuda_lib.device_status(side) == 0
