"""Cases of the operators for requests that share prompts and verify drafts, for timing and for comparing their outputs.

  prefix   attention of requests in groups that share a cached prefix: the prefix is read once per group
  verify   drafted token trees against the target's probabilities, from given random numbers
  compact  keys and values of the accepted nodes to the first places behind the context
  fork     a step of the page ledger: dropped requests freed, others forked onto their rows, grown, and the pages
           that fork could not share copied

``own`` False computes them in plain torch operations (fp32, one rounding at the end; fp64 where sums are compared
with random numbers); True calls paged_kv_prefill_gb300.  ``exact`` computes them in fp64, or one by one in Python,
from their definitions.  All inputs are made on the GPU from the seed; lengths and page tables' sizes follow from the
case alone.
"""
import math
import random

import torch

# whether run() calls the framework
own = False

E4M3 = torch.float8_e4m3fn
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # eight samples of one prompt, a few tokens in: latency
        dict(name="prefix_samples", op="prefix", lens=21, groups=1, reqs_lo=8, reqs_hi=8, new_lo=1, new_hi=1,
             prefix_lo=2048, prefix_hi=2048, own_lo=1, own_hi=64, heads=32, kv_heads=8, dim=128, page=32, layout="HND",
             cache="bf16", sinks=False),
        # a serving batch behind one long system prompt, one token each
        dict(name="prefix_batch", op="prefix", lens=22, groups=1, reqs_lo=64, reqs_hi=64, new_lo=1, new_hi=1,
             prefix_lo=16384, prefix_hi=16384, own_lo=64, own_hi=1024, heads=32, kv_heads=8, dim=128, page=32,
             layout="HND", cache="bf16", sinks=False),
        # several prompts, some sampled often and some hardly, an e4m3 cache, attention sinks
        dict(name="prefix_groups", op="prefix", lens=23, groups=8, reqs_lo=3, reqs_hi=24, new_lo=1, new_hi=1,
             prefix_lo=1500, prefix_hi=9000, own_lo=1, own_hi=2048, heads=64, kv_heads=8, dim=128, page=64,
             layout="NHD", cache="e4m3", sinks=True),
        # questions of 16 to 64 tokens about one document, short heads: compute
        dict(name="prefix_questions", op="prefix", lens=24, groups=1, reqs_lo=16, reqs_hi=16, new_lo=16, new_hi=64,
             prefix_lo=32768, prefix_hi=32768, own_lo=64, own_hi=128, heads=32, kv_heads=8, dim=64, page=16,
             layout="HND", cache="bf16", sinks=False),
        # one request's small tree of likeliest tokens: latency
        dict(name="verify_one", op="verify", lens=31, batch=1, nodes_lo=8, nodes_hi=8, vocab=32000, width=3, draft=False),
        # a batch of such trees
        dict(name="verify_trees", op="verify", lens=32, batch=32, nodes_lo=9, nodes_hi=32, vocab=131072, width=4,
             draft=False),
        # trees drawn from the draft's probabilities: every refusal takes a pass over two rows
        dict(name="verify_drawn", op="verify", lens=33, batch=64, nodes_lo=4, nodes_hi=8, vocab=131072, width=2,
             draft=True),
        # accepted nodes of a small batch: latency
        dict(name="compact_step", op="compact", lens=41, batch=8, nodes_lo=8, nodes_hi=8, path=5, kv_lo=500, kv_hi=4000,
             kv_heads=8, dim=128, page=32, layout="HND", cache="bf16"),
        # a large batch with wide trees and deep paths, an e4m3 cache with a scale per row
        dict(name="compact_wide", op="compact", lens=42, batch=256, nodes_lo=48, nodes_hi=64, path=24, kv_lo=500,
             kv_hi=1500, kv_heads=8, dim=128, page=64, layout="NHD", cache="scaled"),
        # a beam step of one request: latency
        dict(name="fork_beams", op="fork", lens=51, parents=2, children=4, len_lo=1500, len_hi=2500, grow=1, pages=2000,
             kv_heads=8, dim=128, page=32, layout="HND", cache="bf16"),
        # sixteen samples of each of sixteen prompts
        dict(name="fork_samples", op="fork", lens=52, parents=16, children=256, len_lo=1000, len_hi=4000, grow=32,
             pages=5000, kv_heads=8, dim=128, page=32, layout="HND", cache="bf16"),
        # long prompts in large e4m3 pages with a scale per row
        dict(name="fork_long", op="fork", lens=53, parents=8, children=120, len_lo=8000, len_hi=20000, grow=200,
             pages=4500, kv_heads=8, dim=128, page=64, layout="NHD", cache="scaled"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "verify", "compact", "fork"])
    lens = rng.randrange(1 << 30)
    kvh = rng.choice([1, 2, 4, 8])
    if op == "prefix":
        groups = _log_int(rng, 1, 8)
        reqs = _log_int(rng, 1, 32 // groups)
        new = rng.choice([1, 1, 1, 3, 17])
        prefix, tail = _log_int(rng, 1, 12000), _log_int(rng, new, 1500)
        dim = rng.choice([64, 128, 128])
        return dict(op=op, lens=lens, groups=groups, reqs_lo=max(1, reqs // 3), reqs_hi=reqs, new_lo=1, new_hi=new,
                    prefix_lo=max(1, prefix // 3), prefix_hi=prefix, own_lo=max(1, tail // 8), own_hi=tail,
                    heads=kvh * rng.choice([1, 2, 4, 5, 8]), kv_heads=kvh, dim=dim, page=rng.choice([8, 16, 32, 64, 128]),
                    layout=rng.choice(["HND", "NHD"]), cache=rng.choice(["bf16", "e4m3"]) if dim == 128 else "bf16",
                    sinks=rng.choice([False, True]))
    if op == "verify":
        draft = rng.choice([False, True])
        nodes = _log_int(rng, 1, 24 if draft else 64)
        return dict(op=op, lens=lens, batch=_log_int(rng, 1, 16), nodes_lo=max(1, nodes // 2), nodes_hi=nodes,
                    vocab=_log_int(rng, 100, 131072), width=rng.choice([1, 2, 3]), draft=draft)
    page, dim, layout = rng.choice([8, 16, 32, 64]), rng.choice([64, 80, 96, 128]), rng.choice(["HND", "NHD"])
    cache = rng.choice(["bf16", "scaled", "e4m3"])
    if op == "compact":
        nodes = _log_int(rng, 1, 64)
        return dict(op=op, lens=lens, batch=_log_int(rng, 1, 64), nodes_lo=max(1, nodes // 2), nodes_hi=nodes,
                    path=_log_int(rng, 1, nodes), kv_lo=nodes, kv_hi=_log_int(rng, nodes, 1500), kv_heads=kvh, dim=dim,
                    page=page, layout=layout, cache=cache)
    long = _log_int(rng, 1, 4000)
    parents = _log_int(rng, 1, 12)
    children = _log_int(rng, 1, 120)
    grow = rng.choice([0, 1, 40])
    pages = (parents + 2) * (-(-long // page) + 1) + children * (3 + 2 * (-(-grow // page)))
    return dict(op=op, lens=lens, parents=parents, children=children, len_lo=max(1, long // 3), len_hi=long, grow=grow,
                pages=pages + _log_int(rng, 1, 500), kv_heads=kvh, dim=dim, page=page, layout=layout, cache=cache)


# ---------------------------------------------------------------- inputs

def _pool_shape(case, pages):
    k, p = case["kv_heads"], case["page"]
    return (pages, k, p, case["dim"]) if case["layout"] == "HND" else (pages, p, k, case["dim"])


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).to(DEV)


def _sums(n):
    return [sum(n[:i]) for i in range(len(n) + 1)]


def _prefix_lens(case):
    """(requests of each group, prefix lengths, new tokens and own keys of each request): by the case alone."""
    r = random.Random(case["lens"])
    reqs = [r.randint(case["reqs_lo"], case["reqs_hi"]) for _ in range(case["groups"])]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in reqs]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(sum(reqs))]
    return reqs, prefix, new, [max(n, r.randint(case["own_lo"], case["own_hi"])) for n in new]


def _tree_lens(case):
    r = random.Random(case["lens"])
    n = [r.randint(case["nodes_lo"], case["nodes_hi"]) for _ in range(case["batch"])]
    return n, [max(x, r.randint(case["kv_lo"], case["kv_hi"])) for x in n] if "kv_lo" in case else None


def _accepted(case):
    """Accepted nodes of each request.  Some are in their places already; the others come from behind all places that
    are written, so that a second pass moves the same rows again."""
    n, _ = _tree_lens(case)
    r = random.Random(case["lens"] + 1)
    out = []
    for m in n:
        count = r.randint(1, min(case["path"], m))
        stay = r.randint(max(1, 2 * count - m), count)
        out.append(list(range(stay)) + sorted(r.sample(range(count, m), count - stay)))
    return out


def _fork_lens(case):
    """(parents' lengths, which parent each child had, and had taken how much of, which it gets, tokens it grows by)."""
    r = random.Random(case["lens"])
    size = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["parents"])]
    kids = case["children"]
    had = [r.randrange(len(size)) for _ in range(kids)]
    took = [r.randint(1, size[p]) for p in had]
    gets = [r.randrange(len(size)) for _ in range(kids)]
    return size, had, took, gets, [r.randint(0, case["grow"]) for _ in range(kids)]


def _table(rows, order, width):
    """Page tables: the next len(row) pages of `order` for each row of page counts."""
    ends = _sums(rows)
    table = torch.zeros((len(rows), max(width, 1)), dtype=torch.int32, device=DEV)
    for i, u in enumerate(rows):
        table[i, :u] = order[ends[i] : ends[i] + u]
    return table


def _fill_pools(case, pages, g):
    """(pools, scales or None)."""
    shape = _pool_shape(case, pages)
    if case["cache"] == "scaled":
        codes = [torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8).view(E4M3) for _ in "kv"]
        return tuple(codes), tuple(
            torch.exp2(torch.randint(-12, -4, shape[:-1], generator=g, device=DEV).float()) for _ in "kv")
    x = [torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv"]
    return tuple((y.float() * 64).to(E4M3) if case["cache"] == "e4m3" else y for y in x), None


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "prefix":
        reqs, prefix, new, tail = _prefix_lens(case)
        h, d, p = case["heads"], case["dim"], case["page"]
        s["bmm1"], s["bmm2"] = 1.0 / math.sqrt(d), 1.0
        if case["cache"] == "e4m3":
            s["bmm1"], s["bmm2"] = s["bmm1"] / 64, 1.0 / 64
        shared, mine = [-(-x // p) for x in prefix], [-(-x // p) for x in tail]
        pages = sum(shared) + sum(mine) + 4
        s["pools"], _ = _fill_pools(case, pages, g)
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["prefix_table"] = _table(shared, order, max(shared))
        s["table"] = _table(mine, order[sum(shared) :], max(mine))
        s["prefix_lens"], s["seq"] = _ints(prefix), _ints(tail)
        s["cum_groups"], s["cum_q"] = _ints(_sums(reqs)), _ints(_sums(new))
        s["q"] = torch.randn((sum(new), h, d), generator=g, device=DEV).to(torch.bfloat16)
        s["sinks"] = torch.randn(h, generator=g, device=DEV) if case["sinks"] else None
        # what a scheduler knows of its batch
        s["max_q"], s["max_prefix"], s["max_kv"] = max(new), max(prefix), max(tail)
        ends = _sums(new)
        s["max_group_q"] = max(ends[b] - ends[a] for a, b in zip(_sums(reqs), _sums(reqs)[1:]))
        return s
    if case["op"] == "verify":
        n, _ = _tree_lens(case)
        t, vocab = sum(n), case["vocab"]
        r = random.Random(seed)
        parents = []
        for m in n:
            kids, p = [0] * m, [-1]
            for i in range(1, m):
                # breadth first, at most `width` children each
                open_ = [j for j in range(max(0, i - 2 * case["width"]), i) if kids[j] < case["width"]]
                p.append(r.choice(open_[:2]))
                kids[p[-1]] += 1
            parents += p
        s["parents"] = _ints(parents)
        s["cum_q"], s["max_q"] = _ints(_sums(n)), max(n)
        up = (s["parents"].long() + s["cum_q"][:-1].long().repeat_interleave(torch.tensor(n, device=DEV))).clamp(min=0)
        # a draft that knows the target roughly
        z = torch.randn((t, vocab), generator=g, device=DEV) * 6
        s["target"] = torch.softmax(z + torch.randn((t, vocab), generator=g, device=DEV), -1)
        if case["draft"]:
            s["draft"] = torch.softmax(z, -1)
            noise = -torch.log(-torch.log(torch.rand((t, vocab), generator=g, device=DEV).clamp(1e-20, 1 - 1e-7)))
            s["tokens"] = (z[up] + noise).argmax(-1).to(torch.int32)  # drawn from the parents' draft rows
        else:
            s["draft"] = None
            kids = torch.topk(z, min(case["width"], vocab), -1).indices  # the draft's likeliest tokens
            same = (up[:, None] == up[None]) & (torch.arange(t, device=DEV)[None] < torch.arange(t, device=DEV)[:, None])
            same &= s["parents"][None] >= 0
            s["tokens"] = kids[up, same.sum(1).clamp(max=kids.shape[1] - 1)].to(torch.int32)
        s["uniforms"] = torch.rand(t, generator=g, device=DEV)
        s["last"] = torch.rand(len(n), generator=g, device=DEV)
        return s
    if case["op"] == "compact":
        n, kv = _tree_lens(case)
        used = [-(-x // case["page"]) for x in kv]
        pages = sum(used) + 4
        s["pools"], s["scales"] = _fill_pools(case, pages, g)
        s["table"] = _table(used, torch.randperm(pages, generator=g, device=DEV).to(torch.int32), max(used))
        s["seq"], s["cum_q"] = _ints(kv), _ints(_sums(n))
        taken = _accepted(case)
        s["accepted"] = _ints([x + [-1] * (max(n) - len(x)) for x in taken])
        s["count"] = _ints([len(x) for x in taken])
        return s
    size, had, took, gets, grow = _fork_lens(case)
    p, pages, first = case["page"], case["pages"], len(size)
    s["pools"], s["scales"] = _fill_pools(case, pages, g)
    width = max(-(-(max(size) + case["grow"]) // p), 1)
    r = random.Random(seed)
    order = r.sample(range(pages), pages)
    rows, at = [], 0
    for x in size:
        u = -(-x // p)
        rows.append(order[at : at + u])
        at += u
    for parent, x in zip(had, took):
        # a fork of an earlier step: whole pages shared, a page of its own behind them
        row = rows[parent][: x // p]
        if x % p:
            row = row + [order[at]]
            at += 1
        rows.append(row)
    refs = [0] * pages
    for row in rows:
        for x in row:
            refs[x] += 1
    s["table"] = _ints([row + [0] * (width - len(row)) for row in rows])
    s["refs"], s["seq"] = _ints(refs), _ints(size + took)
    s["children"] = _ints(range(first, first + len(gets)))
    s["parents"] = _ints(gets)
    s["to"] = _ints([size[x] + y for x, y in zip(gets, grow)])
    return s


# ---------------------------------------------------------------- the plain forms

def _keys(s, pool, table):
    """[rows, kv heads, keys, dim] in fp32 of a pool, through a page table."""
    x = pool.view(torch.uint8)[table.long()].view(E4M3) if pool.dtype == E4M3 else pool[table.long()]
    x = x.float()
    x = x.transpose(2, 3) if s["case"]["layout"] == "HND" else x
    return x.flatten(1, 2).transpose(1, 2)


def _scores(s, first, count, width, table, sees):
    """Scores [rows, kv heads, heads of one, width, keys] of `width` query rows from `first` on against the keys of a
    table, unseen ones at -inf."""
    c = s["case"]
    k = _keys(s, s["pools"][0], table)
    row = (first[:, None] + torch.arange(width, device=DEV)).clamp(max=s["q"].shape[0] - 1)
    n, hk, d = len(first), c["kv_heads"], c["dim"]
    q = s["q"][row].float().view(n, width, hk, -1, d).permute(0, 2, 3, 1, 4)
    x = (q.reshape(n, hk, -1, d) @ k.transpose(2, 3)).mul_(s["bmm1"]).view(n, hk, -1, width, k.shape[2])
    x.masked_fill_(~sees(torch.arange(width, device=DEV)[None, :, None], torch.arange(k.shape[2], device=DEV))[:, None, None],
                   -math.inf)
    return x, row, torch.arange(width, device=DEV)[None] < count[:, None]


def _weigh(s, x, row, real, top, pool, table):
    """Sums of exponentials [tokens, heads] and of weighted values [tokens, heads, dim]."""
    c = s["case"]
    n, hk, grp, width = x.shape[:4]
    x.sub_(top[row].permute(0, 2, 1).reshape(n, hk, grp, width, 1)).exp_()
    o = x.view(n, hk, grp * width, -1) @ _keys(s, pool, table)
    o = o.view(n, c["heads"], width, c["dim"]).transpose(1, 2)[real]
    return x.sum(-1).view(n, c["heads"], width).transpose(1, 2)[real], o


def _plain_prefix(s):
    c = s["case"]
    cum, groups = s["cum_q"].long(), s["cum_groups"].long()
    starts = cum[groups]
    new, seq = (cum[1:] - cum[:-1]), s["seq"].long()
    lens = s["prefix_lens"].long()
    xp, rp, real_p = _scores(s, starts[:-1], starts[1:] - starts[:-1], s["max_group_q"], s["prefix_table"],
                             lambda i, j: (j < lens[:, None, None]).expand(-1, i.shape[1], -1))
    xo, ro, real_o = _scores(s, cum[:-1], new, s["max_q"], s["table"], lambda i, j: j <= (seq - new)[:, None, None] + i)

    def tops(x, real):
        return x.amax(-1).view(len(x), c["heads"], -1).transpose(1, 2)[real]

    top = torch.maximum(tops(xp, real_p), tops(xo, real_o))
    den_p, out_p = _weigh(s, xp, rp, real_p, top, s["pools"][1], s["prefix_table"])
    den_o, out_o = _weigh(s, xo, ro, real_o, top, s["pools"][1], s["table"])
    den = den_p + den_o
    if s["sinks"] is not None:
        den = den + torch.exp(s["sinks"] - top)
    return ((out_p + out_o) / den[..., None] * s["bmm2"]).to(torch.bfloat16)


def _plain_verify(s):
    """All nodes at once: whether each would be taken, were its parent on the path; then the path, then the last token."""
    cum, tokens, vocab = s["cum_q"].long(), s["tokens"].long(), s["case"]["vocab"]
    t, b = len(tokens), len(cum) - 1
    at = torch.arange(t, device=DEV)
    req = torch.searchsorted(cum[1:], at, right=True)
    root = s["parents"] < 0
    up = torch.where(root, at, s["parents"].long() + cum[req])
    before = (up[:, None] == up[None]) & (at[None] < at[:, None]) & ~root[None] & ~root[:, None]  # earlier siblings
    p, u = s["target"][up, tokens].double(), s["uniforms"].double()
    if s["draft"] is None:
        twin = before & (tokens[None] == tokens[:, None])
        again = twin.any(1)
        mass = 1 - ((before & ~again[None]) * p[None]).sum(1)
        takes = (u * mass < p) & ~again & ~root
    else:
        q = s["draft"][up, tokens].double()
        rank = before.sum(1)
        a = torch.zeros(t, dtype=torch.float64, device=DEV)  # of each node's children so far
        mass = torch.ones_like(a)
        takes = torch.zeros(t, dtype=torch.bool, device=DEV)
        kids = torch.zeros(t, dtype=torch.long, device=DEV).index_add_(0, up[~root], torch.ones_like(up[~root]))
        for k in range(s["case"]["width"]):  # what the k-th child finds depends on what the one before it left
            rest = (p - a[up] * q).clamp(min=0)
            takes |= (rank == k) & (u * q * mass[up] < rest) & ~root
            a = torch.where(kids > k, a + mass, a)
            mass = (s["target"].double() - a[:, None] * s["draft"].double()).clamp_(min=0).sum(1)
    chosen = takes & ~(before & takes[None]).any(1)
    # a node is on the path if it and all above it are chosen: seen by squaring the parents' relation
    above = (up[:, None] == at[None]) & ~root[:, None]
    reach = (above | (at[:, None] == at[None])).double()
    reach = (reach @ reach).clamp_(max=1)
    reach = (reach @ reach).clamp_(max=1)
    reach = (reach @ reach).clamp_(max=1)
    reach = (reach @ reach).clamp_(max=1)
    reach = (reach @ reach).clamp_(max=1)
    reach = (reach @ reach).clamp_(max=1)  # paths of up to 64 nodes
    path = (reach @ (~(chosen | root)).double()[:, None])[:, 0] == 0
    count = torch.zeros(b, dtype=torch.long, device=DEV).index_add_(0, req[path], torch.ones_like(req[path]))
    accepted = torch.full((b, s["max_q"]), -1, dtype=torch.int32, device=DEV)
    rank = torch.cumsum(path, 0) - 1 - (torch.cumsum(count, 0) - count)[req]
    accepted[req[path], rank[path]] = (at - cum[req])[path].int()
    end = cum[:-1] + accepted[torch.arange(b, device=DEV), count - 1]
    whole = s["target"][end].double()
    if s["draft"] is None:
        rest = whole.clone()
        out = (up[None] == end[:, None]) & ~root[None]
        who, node = out.nonzero(as_tuple=True)
        rest[who, tokens[node]] = 0
    else:
        rest = (whole - a[end, None] * s["draft"][end].double()).clamp_(min=0)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, whole)
    run_ = torch.cumsum(rest, 1)
    first = (run_ <= s["last"].double()[:, None] * run_[:, -1:]).sum(1)
    last = vocab - 1 - (rest.flip(1) > 0).int().argmax(1)
    return accepted, count.int(), torch.minimum(first, last).int()


def _slots(s, pool):
    """The pool as [pages, page, heads, ...], to be indexed by (page, slot)."""
    x = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
    return x.transpose(1, 2) if s["case"]["layout"] == "HND" else x


def _caches(s):
    return (*s["pools"], *(s["scales"] or ()))


def _plain_compact(s):
    p = s["case"]["page"]
    n = (s["cum_q"][1:] - s["cum_q"][:-1]).long()
    ctx = (s["seq"].long() - n)[:, None]
    i = torch.arange(s["accepted"].shape[1], device=DEV)[None]
    moves = i < s["count"][:, None]
    b = torch.arange(len(n), device=DEV)[:, None].expand_as(moves)[moves]
    to, frm = (ctx + i)[moves], (ctx + s["accepted"].long())[moves]
    table = s["table"].long()

    def move(x):
        x[table[b, to // p], to % p] = x[table[b, frm // p], frm % p]

    k, v, *scales = (_slots(s, x) for x in _caches(s))
    move(k)
    move(v)
    if scales:
        move(scales[0])
        move(scales[1])
    return (*_caches(s), (ctx[:, 0] + s["count"]).int())


def _plain_fork(s):
    table, refs, seq, p = s["table"], s["refs"], s["seq"], s["case"]["page"]
    kids, parents = s["children"].long(), s["parents"].long()
    col = torch.arange(table.shape[1], device=DEV)[None]
    held = col < (-(-seq[kids].long() // p))[:, None]
    pages = table[kids][held].long()
    refs.index_add_(0, pages, -torch.ones_like(pages, dtype=torch.int32))
    # fork: whole pages shared, one of its own for what is left
    size = seq[parents].long()
    whole = col < (size // p)[:, None]
    rows = table[parents]
    table[kids] = torch.where(whole, rows, table[kids])
    pages = rows[whole].long()
    refs.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    part = size % p != 0
    free = (refs == 0).nonzero()[:, 0].int()
    rank = torch.cumsum(part, 0) - 1
    src = torch.where(part, rows.gather(1, (size // p).clamp(max=table.shape[1] - 1)[:, None])[:, 0], -1)
    dst = torch.where(part, free[rank.clamp(min=0)], -1)
    table[kids[part], (size // p)[part]] = dst[part]
    refs[dst[part].long()] = 1
    seq[kids] = seq[parents]
    # grow: pages for the tokens that come
    old, new = -(-size // p), -(-s["to"].long() // p)
    fresh = (col >= old[:, None]) & (col < new[:, None])
    free = (refs == 0).nonzero()[:, 0].int()
    got = free[: int((new - old).sum())]
    grown = table[kids]
    grown[fresh] = got
    table[kids] = grown
    refs[got.long()] = 1
    seq[kids] = s["to"]
    on = part
    a, b = src[on].long(), dst[on].long()

    def copy(x):
        y = x.view(torch.uint8) if x.dtype == E4M3 else x
        y[b] = y[a]

    k, v, *scales = _caches(s)
    copy(k)
    copy(v)
    if scales:
        copy(scales[0])
        copy(scales[1])
    return (table, seq, refs, src.int(), dst.int(), *_caches(s))


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"prefix": _plain_prefix, "verify": _plain_verify, "compact": _plain_compact, "fork": _plain_fork}[op](s)
    import paged_kv_prefill_gb300 as b2pa

    c = s["case"]
    if op == "prefix":
        return b2pa.prefix_attention(s["q"], s["pools"], s["prefix_table"], s["prefix_lens"], s["cum_groups"], s["table"],
                                     s["seq"], s["max_q"], s["max_prefix"], s["max_kv"], s["bmm1"], s["bmm2"], s["cum_q"],
                                     max_group_q_len=s["max_group_q"], kv_layout=c["layout"], sinks=s["sinks"])
    if op == "verify":
        return b2pa.verify_trees(s["target"], s["tokens"], s["parents"], s["uniforms"], s["last"], s["max_q"],
                                 s["cum_q"], draft_probs=s["draft"])
    if op == "compact":
        lens = b2pa.compact_kv(s["pools"], s["table"], s["seq"], s["cum_q"], s["accepted"], s["count"],
                               kv_scales=s["scales"], kv_layout=c["layout"])
        return (*_caches(s), lens)
    b2pa.free_pages(s["table"], s["seq"], s["refs"], s["children"], c["page"])
    src, dst = b2pa.fork_pages(s["table"], s["seq"], s["refs"], s["parents"], s["children"], c["page"])
    b2pa.grow_pages(s["table"], s["seq"], s["refs"], s["children"], s["to"], c["page"])
    b2pa.copy_pages(s["pools"], src, dst, kv_scales=s["scales"], kv_layout=c["layout"])
    return (s["table"], s["seq"], s["refs"], src, dst, *_caches(s))


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(case):
    """One token's keys and values of all heads."""
    e, s = (2, 0) if case["cache"] == "bf16" else (1, 4 if case["cache"] == "scaled" else 0)
    return 2 * case["kv_heads"] * (case["dim"] * e + s)


def work(case):
    op = case["op"]
    if op == "prefix":
        reqs, prefix, new, tail = _prefix_lens(case)
        d, h, p = case["dim"], case["heads"], case["page"]
        ends = _sums(reqs)
        pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, tail))
        pairs += sum(sum(new[a:b]) * x for a, b, x in zip(ends, ends[1:], prefix))
        b = (sum(prefix) + sum(tail)) * _row_bytes(case) + sum(new) * h * d * 4
        return dict(bytes=b + 4 * sum(-(-x // p) for x in prefix + tail), flops=4 * d * h * pairs)
    if op == "verify":
        # the last accepted node's row of each request; nodes' tokens, parents, numbers and probabilities
        n, _ = _tree_lens(case)
        rows = (2 if case["draft"] else 1) * case["batch"]
        return dict(bytes=4 * rows * case["vocab"] + 20 * sum(n), flops=2 * rows * case["vocab"])
    if op == "compact":
        moved = sum(sum(i != x for i, x in enumerate(a)) for a in _accepted(case))
        return dict(bytes=2 * moved * _row_bytes(case) + 4 * sum(len(a) for a in _accepted(case)), flops=0)
    size, had, took, gets, grow = _fork_lens(case)
    p = case["page"]
    copies = sum(size[x] % p != 0 for x in gets)
    # freed rows read, parents' rows read once, children's written; counts read, and written where they change
    pages = sum(-(-x // p) for x in took) + sum(-(-size[x] // p) for x in set(gets))
    pages += sum(-(-(size[x] + y) // p) for x, y in zip(gets, grow))
    return dict(bytes=2 * copies * p * _row_bytes(case) + 8 * pages + 4 * case["pages"], flops=0)


# ---------------------------------------------------------------- the definitions, in 64 bits or one by one

def _exact_prefix(case, s):
    reqs, prefix, new, tail = _prefix_lens(case)
    p, hk, grp = case["page"], case["kv_heads"], case["heads"] // case["kv_heads"]

    def rows(pool, table, length):
        used = table[: -(-length // p)].long()
        x = pool.view(torch.uint8)[used].view(E4M3) if pool.dtype == E4M3 else pool[used]
        x = x.to(torch.float64).permute(1, 0, 2, 3) if case["layout"] == "HND" else x.to(torch.float64).permute(2, 0, 1, 3)
        return x.reshape(hk, -1, case["dim"])[:, :length]

    out, row, b = [], 0, 0
    for g, count in enumerate(reqs):
        kp, vp = (rows(x, s["prefix_table"][g], prefix[g]) for x in s["pools"])
        for _ in range(count):
            n, length = new[b], tail[b]
            k, v = (torch.cat([x, rows(y, s["table"][b], length)], 1) for x, y in zip((kp, vp), s["pools"]))
            q = s["q"][row : row + n].double().permute(1, 0, 2).reshape(hk, grp * n, -1)
            x = torch.matmul(q, k.transpose(1, 2)).view(hk * grp, n, -1) * s["bmm1"]
            last = prefix[g] + length - n + torch.arange(n, device=DEV)[:, None]
            x = torch.where(torch.arange(x.shape[2], device=DEV) <= last, x, -math.inf)
            top = x.amax(-1, keepdim=True)
            e = torch.exp(x - top)
            den = e.sum(-1, keepdim=True)
            if s["sinks"] is not None:
                den = den + torch.exp(s["sinks"].double().view(-1, 1, 1) - top)
            o = torch.matmul(e.view(hk, grp * n, -1), v).view(hk * grp, n, -1) / den * s["bmm2"]
            out.append(o.permute(1, 0, 2))
            row += n
            b += 1
    return torch.cat(out)


def _exact_verify(case, s):
    n, _ = _tree_lens(case)
    tokens, parents = s["tokens"].tolist(), s["parents"].tolist()
    uniforms, last = s["uniforms"].tolist(), s["last"].tolist()
    taken, counts, chosen = [], [], []
    at = 0
    for b, m in enumerate(n):
        node, path = 0, [0]
        while True:
            p = s["target"][at + node].double()
            q = s["draft"][at + node].double() if case["draft"] else None
            rest, mass, a, found = p.clone(), 1.0, 0.0, None
            for i in range(1, m):
                if parents[at + i] != node:
                    continue
                x, u = tokens[at + i], uniforms[at + i]
                if u * (float(q[x]) if case["draft"] else 1.0) * mass < float(rest[x]):
                    found = i
                    break
                if case["draft"]:
                    a += mass
                    rest = torch.clamp(p - a * q, min=0)
                    mass = float(rest.sum())
                else:
                    mass -= float(rest[x])
                    rest[x] = 0
            if found is None:
                break
            node = found
            path.append(node)
        if not float(rest.sum()) > 0:
            rest = p
        ends = torch.cumsum(rest, 0)
        over = (ends > last[b] * ends[-1]).nonzero()
        chosen.append(int(over[0]) if len(over) else int(rest.nonzero()[-1]))
        taken.append(path + [-1] * (max(n) - len(path)))
        counts.append(len(path))
        at += m
    return _ints(taken), _ints(counts), _ints(chosen)


def _exact_compact(case, s):
    n, kv = _tree_lens(case)
    p, table = case["page"], s["table"].tolist()
    out = []
    for x in _caches(s):
        x = x.to(torch.float64)
        y = x.transpose(1, 2) if case["layout"] == "HND" else x
        for b, path in enumerate(_accepted(case)):
            ctx = kv[b] - n[b]
            for i, a in enumerate(path):
                if i != a:
                    y[table[b][(ctx + i) // p], (ctx + i) % p] = y[table[b][(ctx + a) // p], (ctx + a) % p]
        out.append(x)
    return (*out, _ints([x - m + len(a) for x, m, a in zip(kv, n, _accepted(case))]))


def _exact_fork(case, s):
    size, had, took, gets, grow = _fork_lens(case)
    table, refs, seq, p = s["table"].tolist(), s["refs"].tolist(), s["seq"].tolist(), case["page"]
    first = len(size)
    for i in range(first, len(seq)):
        for x in table[i][: -(-seq[i] // p)]:
            refs[x] -= 1
    src, dst = [], []
    for parent in gets:  # whole pages first: a page is free when nobody holds it
        for x in table[parent][: size[parent] // p]:
            refs[x] += 1
    free = [i for i, x in enumerate(refs) if x == 0]
    for i, parent in enumerate(gets):
        whole = size[parent] // p
        table[first + i][:whole] = table[parent][:whole]
        part = size[parent] % p != 0
        src.append(table[parent][whole] if part else -1)
        dst.append(free.pop(0) if part else -1)
        if part:
            table[first + i][whole] = dst[-1]
            refs[dst[-1]] = 1
        seq[first + i] = size[parent]
    for i, more in enumerate(grow):
        for col in range(-(-seq[first + i] // p), -(-(seq[first + i] + more) // p)):
            table[first + i][col] = free.pop(0)
            refs[table[first + i][col]] = 1
        seq[first + i] += more
    caches = []
    on = [(a, b) for a, b in zip(src, dst) if a >= 0]
    for x in _caches(s):
        x = x.to(torch.float64)
        if on:
            x[[b for _, b in on]] = x[[a for a, _ in on]]
        caches.append(x)
    return (_ints(table), _ints(seq), _ints(refs), _ints(src), _ints(dst), *caches)


def exact(case, seed):
    s = prepare(case, seed)
    return {"prefix": _exact_prefix, "verify": _exact_verify, "compact": _exact_compact, "fork": _exact_fork}[case["op"]](
        case, s)
