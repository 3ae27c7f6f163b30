"""Cases of the operators around the paged cache, for timing and for comparing their outputs.

Four operators, each as a serving step calls it:
  rope    per-head RMS norm of queries and keys with the rotary rotation (one or several position axes)
  append  new keys and values quantised to e4m3, one power-of-two scale per token and kv head, into the pools
  read    rows of such a cache read back as bf16
  tree    attention of a batch of drafted token trees over a paged cache

``own`` False computes them in plain torch operations (fp32, one rounding at the end); True calls
paged_kv_prefill_gb300.  ``exact`` computes them in fp64 from their definitions.  All inputs are made on the
GPU from the seed; lengths and page tables' sizes follow from the case alone.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 32 requests: latency
        dict(name="rope_step", op="rope", tokens=32, heads=32, kv_heads=8, dim=128, rot=128, axes=1, pairs=False,
             norm=True),
        # the prompt batch of the benchmark workload (11750 tokens)
        dict(name="rope_prompts", op="rope", tokens=11750, heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             pairs=False, norm=True),
        # image and video tokens with (time, height, width) positions
        dict(name="rope_video", op="rope", tokens=16384, heads=64, kv_heads=8, dim=128, rot=128, axes=3,
             pairs=False, norm=True),
        # the cache write of a decoding step
        dict(name="append_step", op="append", tokens=32, kv_heads=8, dim=128, page=32, layout="HND"),
        # the cache write of a long prompt batch
        dict(name="append_prompts", op="append", tokens=32768, kv_heads=8, dim=128, page=64, layout="NHD"),
        # a cached prefix of 2048 tokens restored
        dict(name="read_prefix", op="read", tokens=2048, kv_heads=8, dim=128, page=32, layout="HND"),
        # a batch's whole context restored, short heads
        dict(name="read_context", op="read", tokens=131072, kv_heads=8, dim=64, page=16, layout="NHD"),
        # one request with a small tree: latency
        dict(name="tree_one", op="tree", lens=11, batch=1, nodes_lo=8, nodes_hi=8, kv_lo=2048, kv_hi=2048, heads=32,
             kv_heads=8, dim=128, page=32, layout="HND", cache="bf16", window=-1, sinks=False),
        # a serving batch, ragged trees and contexts
        dict(name="tree_batch", op="tree", lens=12, batch=32, nodes_lo=9, nodes_hi=16, kv_lo=512, kv_hi=8192,
             heads=32, kv_heads=8, dim=128, page=32, layout="HND", cache="bf16", window=-1, sinks=False),
        # wide trees with eight query heads per kv head: 512 rows per kv head
        dict(name="tree_wide", op="tree", lens=13, batch=8, nodes_lo=48, nodes_hi=64, kv_lo=1024, kv_hi=16384,
             heads=64, kv_heads=8, dim=128, page=64, layout="NHD", cache="bf16", window=-1, sinks=False),
        # an e4m3 cache with scales for the whole tensor
        dict(name="tree_e4m3", op="tree", lens=14, batch=32, nodes_lo=5, nodes_hi=8, kv_lo=1024, kv_hi=16384,
             heads=32, kv_heads=8, dim=128, page=32, layout="HND", cache="e4m3", window=-1, sinks=False),
        # a sliding-window layer with attention sinks at head_dim 64
        dict(name="tree_window", op="tree", lens=15, batch=16, nodes_lo=24, nodes_hi=32, kv_lo=600, kv_hi=4096,
             heads=64, kv_heads=8, dim=64, page=16, layout="HND", cache="bf16", window=127, sinks=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "tree", "tree"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([dim, dim, dim // 2])
        kvh = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log_int(rng, 1, 8192), heads=kvh * rng.choice([1, 2, 4, 5, 8]), kv_heads=kvh,
                    dim=dim, rot=rot, axes=rng.choice([1, 1, 2, 3]), pairs=rng.choice([False, True]),
                    norm=rng.choice([True, True, False]))
    if op in ("append", "read"):
        return dict(op=op, tokens=_log_int(rng, 1, 32768), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 80, 96, 128, 256]) if op == "append" else rng.choice([64, 80, 96, 128]),
                    page=rng.choice([8, 16, 32, 64]), layout=rng.choice(["HND", "NHD"]))
    nodes = _log_int(rng, 1, 64)
    kv = max(nodes, _log_int(rng, 64, 8192))
    dim = rng.choice([64, 128, 128])
    kvh = rng.choice([1, 2, 4, 8])
    window = rng.choice([-1, -1, 127, 1000])
    return dict(op=op, lens=rng.randrange(1 << 30), batch=_log_int(rng, 1, 16), nodes_lo=max(1, nodes // 2),
                nodes_hi=nodes, kv_lo=max(nodes, kv // 4), kv_hi=kv, heads=kvh * rng.choice([1, 2, 4, 5, 8]),
                kv_heads=kvh, dim=dim, page=rng.choice([8, 16, 32, 64, 128]), layout=rng.choice(["HND", "NHD"]),
                cache=rng.choice(["bf16", "e4m3"]) if dim == 128 else "bf16", window=window,
                sinks=rng.choice([False, True]))


# ---------------------------------------------------------------- inputs

def _pool_shape(case, pages):
    k, p = case["kv_heads"], case["page"]
    return (pages, k, p, case["dim"]) if case["layout"] == "HND" else (pages, p, k, case["dim"])


def _tree_lens(case):
    """(tree sizes, kv lengths with the trees' own keys) of the batch: by the case alone."""
    r = random.Random(case["lens"])
    n = [r.randint(case["nodes_lo"], case["nodes_hi"]) for _ in range(case["batch"])]
    return n, [max(x, r.randint(case["kv_lo"], case["kv_hi"])) for x in n]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)

    s = dict(case=case)
    if case["op"] == "rope":
        t, h, k, d, rot = (case[x] for x in ("tokens", "heads", "kv_heads", "dim", "rot"))
        # queries and keys are views of one projection's output, as a model has them
        qkv = normal(t, (h + 2 * k) * d, scale=1.5)
        s["q"] = qkv[:, : h * d].view(t, h, d)
        s["k"] = qkv[:, h * d : (h + k) * d].view(t, k, d)
        s["qw"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        s["kw"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        far = 32768
        inv = 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
        ang = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        a = case["axes"]
        if a == 1:
            # requests one after the other, each at its own place in its sequence
            first = torch.randint(0, far // 2, (1 + t // 512,), generator=g, device=DEV)
            at = torch.arange(t, device=DEV)
            s["positions"] = (first[at // 512] + at % 512).to(torch.int32)
            s["axis_of"] = None
        else:
            s["positions"] = torch.randint(0, 512, (a, t), generator=g, device=DEV).to(torch.int32)
            cuts = [round(i * (rot // 2) / a) for i in range(a + 1)]
            s["axis_of"] = [i for i in range(a) for _ in range(cuts[i + 1] - cuts[i])]
        return s
    if case["op"] in ("append", "read"):
        t, k, d, p = (case[x] for x in ("tokens", "kv_heads", "dim", "page"))
        pages = (t + t // 4) // p + 1
        shape = _pool_shape(case, pages)
        if t < 512:  # a decoding step: every token at its own request's place
            s["loc"] = torch.randperm(pages * p, generator=g, device=DEV)[:t].to(torch.int32)
        else:  # prompts: whole pages, anywhere in the pool
            at = torch.arange(t, device=DEV)
            s["loc"] = (torch.randperm(pages, generator=g, device=DEV)[at // p] * p + at % p).to(torch.int32)
        # the pools start as other requests left them
        codes = [torch.randint(0, 127, shape, generator=g, device=DEV, dtype=torch.uint8).view(E4M3) for _ in "kv"]
        s["pools"] = tuple(codes)
        s["scales"] = tuple(
            torch.exp2(torch.randint(-12, -4, shape[:-1], generator=g, device=DEV).float()) for _ in "kv")
        if case["op"] == "append":
            # rows of very different sizes: what the scale of each row is for
            s["k_new"], s["v_new"] = (
                (torch.randn((t, k, d), generator=g, device=DEV)
                 * torch.exp2(3 * torch.randn((t, k, 1), generator=g, device=DEV))).to(torch.bfloat16) for _ in "kv")
        return s
    n, kv = _tree_lens(case)
    b, h, k, d, p = (case[x] for x in ("batch", "heads", "kv_heads", "dim", "page"))
    used = [-(-x // p) for x in kv]
    pages = sum(used) + 4
    shape = _pool_shape(case, pages)
    pools = [normal(*shape) for _ in "kv"]
    s["bmm1"], s["bmm2"] = 1.0 / math.sqrt(d), 1.0
    if case["cache"] == "e4m3":
        pools = [(x.float() * 64).to(E4M3) for x in pools]
        s["bmm1"], s["bmm2"] = s["bmm1"] / 64, 1.0 / 64
    s["pools"] = tuple(pools)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((b, max(used)), dtype=torch.int32, device=DEV)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at : at + u]
        at += u
    s["table"] = table
    s["q"] = normal(sum(n), h, d)
    s["seq"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["cum_q"] = torch.tensor([sum(n[:i]) for i in range(b + 1)], dtype=torch.int32, device=DEV)
    s["max_q"], s["max_kv"] = case["nodes_hi"], max(case["kv_hi"], max(kv))
    s["sinks"] = torch.randn(h, generator=g, device=DEV) if case["sinks"] else None
    # each node hangs on an earlier node or on the context's last token
    r = random.Random(seed)
    words = -(-case["nodes_hi"] // 32)
    rows, pos = [], []
    for m, length in zip(n, kv):
        seen, depth = [], []
        for i in range(m):
            up = r.randint(-1, i - 1)
            seen.append((1 << i) | (seen[up] if up >= 0 else 0))
            depth.append(depth[up] + 1 if up >= 0 else 0)
        rows += [[((x >> 32 * w) & 0xFFFFFFFF) for w in range(words)] for x in seen]
        pos += [length - m + x for x in depth]
    bits = torch.tensor(rows, dtype=torch.int64).view(-1, words)
    s["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).to(DEV)
    s["positions"] = torch.tensor(pos, dtype=torch.int32).to(DEV)
    return s


# ---------------------------------------------------------------- the plain forms

def _rms(x, w, eps):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _turn(x, cos, sin, pairs):
    rot = 2 * cos.shape[-1]
    c, n = cos[:, None], sin[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., : rot // 2], x[..., rot // 2 : rot])
    u, v = a * c - b * n, b * c + a * n
    both = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([both, x[..., rot:]], -1).to(torch.bfloat16)


def _plain_rope(s):
    half = s["cos_sin"].shape[1] // 2
    pos = s["positions"].long()
    if s["axis_of"] is None:
        cos, sin = s["cos_sin"][pos, :half], s["cos_sin"][pos, half:]
    else:
        at = pos[torch.tensor(s["axis_of"], device=DEV)].t()
        i = torch.arange(half, device=DEV)
        cos, sin = s["cos_sin"][at, i], s["cos_sin"][at, half + i]
    pairs = s["case"]["pairs"]
    q = _turn(_rms(s["q"].float(), s["qw"], 1e-6), cos, sin, pairs)
    k = _turn(_rms(s["k"].float(), s["kw"], 1e-6), cos, sin, pairs)
    return q, k


def _slots(s, pool):
    """The pool as [pages, page, heads, ...], and (page, slot) of each token."""
    loc, p = s["loc"].long(), s["case"]["page"]
    return (pool.transpose(1, 2) if s["case"]["layout"] == "HND" else pool), loc // p, loc % p


def _plain_append(s):
    def write(new, pool, scales):
        x = new.float()
        top, e = torch.frexp(x.abs().amax(-1))
        # the smallest power of two that brings the row's largest value to 448 = 0.875 * 2^9 at most
        e = torch.where(top == 0, 0, torch.where(top <= 0.875, e - 9, e - 8))
        scale = torch.ldexp(torch.ones_like(top), e)
        at, page, slot = _slots(s, pool.view(torch.uint8))
        at[page, slot] = (x / scale[..., None]).to(E4M3).view(torch.uint8)
        _slots(s, scales)[0][page, slot] = scale

    write(s["k_new"], s["pools"][0], s["scales"][0])
    write(s["v_new"], s["pools"][1], s["scales"][1])
    return *s["pools"], *s["scales"]


def _plain_read(s):
    def back(pool, scales):
        at, page, slot = _slots(s, pool.view(torch.uint8))
        codes = at[page, slot].view(E4M3).float()
        return (codes * _slots(s, scales)[0][page, slot][..., None]).to(torch.bfloat16)

    return back(s["pools"][0], s["scales"][0]), back(s["pools"][1], s["scales"][1])


def _sees(s, keys, width):
    """[batch, width, keys]: whether node i of a request sees key j; and the rows' places in the query."""
    c = s["case"]
    first, n = s["cum_q"][:-1].long(), (s["cum_q"][1:] - s["cum_q"][:-1]).long()
    ctx = s["seq"].long() - n
    i, j = torch.arange(width, device=DEV), torch.arange(keys, device=DEV)
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    node = j[None] - ctx[:, None]
    at = node.clamp(0, 32 * s["mask"].shape[1] - 1)
    word = torch.gather(s["mask"][row].long(), 2, (at // 32)[:, None].expand(-1, width, -1))
    sees = ((word >> (at % 32)[:, None]) & 1 == 1) & (node >= 0)[:, None] & (node < n[:, None])[:, None]
    old = (node < 0)[:, None]
    if c["window"] >= 0:
        old = old & (j >= s["positions"][row].long()[..., None] - c["window"])
    return sees | old, row, i[None] < n[:, None]


def _cache_rows(s, pool):
    """[batch, heads, keys, dim] in fp32 of a pool, through the page table."""
    x = pool.view(torch.uint8)[s["table"].long()].view(E4M3) if pool.dtype == E4M3 else pool[s["table"].long()]
    x = x.float()
    x = x.transpose(2, 3) if s["case"]["layout"] == "HND" else x
    return x.flatten(1, 2).transpose(1, 2)


def _plain_tree(s):
    c = s["case"]
    k, v = _cache_rows(s, s["pools"][0]), _cache_rows(s, s["pools"][1])
    sees, row, real = _sees(s, k.shape[2], s["max_q"])
    b, w, hk, d = c["batch"], s["max_q"], c["kv_heads"], c["dim"]
    grp = c["heads"] // hk
    q = s["q"][row].float().view(b, w, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hk, grp * w, d)
    x = (q @ k.transpose(2, 3)).mul_(s["bmm1"]).view(b, hk, grp, w, -1)
    x.masked_fill_(~sees[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    e = x.sub_(top).exp_()
    den = e.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        den = den + torch.exp(s["sinks"].view(1, hk, grp, 1, 1) - top)
    o = (e.view(b, hk, grp * w, -1) @ v).view(b, hk, grp, w, d) / den * s["bmm2"]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, w, c["heads"], d)
    return o[real].to(torch.bfloat16)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "tree": _plain_tree}[op](s)
    import paged_kv_prefill_gb300 as b2pa

    c = s["case"]
    if op == "rope":
        return b2pa.qk_norm_rope(s["q"], s["k"], s["cos_sin"], s["positions"], s["qw"], s["kw"], eps=1e-6,
                                 axis_of=s["axis_of"], interleaved=c["pairs"])
    if op == "append":
        b2pa.append_kv_scaled(s["k_new"], s["v_new"], s["pools"], s["scales"], s["loc"], kv_layout=c["layout"])
        return *s["pools"], *s["scales"]
    if op == "read":
        return b2pa.read_kv_scaled(s["pools"], s["scales"], s["loc"], kv_layout=c["layout"])
    return b2pa.tree_attention(s["q"], s["pools"], s["table"], s["seq"], s["mask"], s["max_q"], s["max_kv"],
                               s["bmm1"], s["bmm2"], s["cum_q"],
                               positions=s["positions"] if c["window"] >= 0 else None, window_left=c["window"],
                               kv_layout=c["layout"], sinks=s["sinks"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "rope":
        t, rows = case["tokens"], case["tokens"] * (case["heads"] + case["kv_heads"])
        d = case["dim"]
        table = 4 * min(t * case["rot"], 32768 * case["rot"])
        return dict(bytes=2 * rows * d * 2 + 4 * t * case["axes"] + table + 4 * d, flops=rows * (4 * d + 3 * case["rot"]))
    if op in ("append", "read"):
        n = 2 * case["tokens"] * case["kv_heads"]
        return dict(bytes=n * case["dim"] * 3 + 4 * n + 4 * case["tokens"], flops=2 * n * case["dim"])
    n, kv = _tree_lens(case)
    d, h, k, w = case["dim"], case["heads"], case["kv_heads"], case["window"]
    ctx = [x - m if w < 0 else min(x - m, w) for m, x in zip(n, kv)]
    size = 1 if case["cache"] == "e4m3" else 2
    b = sum(c + m for c, m in zip(ctx, n)) * k * d * 2 * size + sum(n) * h * d * 4 + 4 * sum(n) * -(-max(n) // 32)
    b += 4 * sum(-(-x // case["page"]) for x in kv)
    return dict(bytes=b, flops=4 * d * h * sum(m * (c + 1) for c, m in zip(ctx, n)))


# ---------------------------------------------------------------- the definitions in 64 bits

def _nearest_e4m3(x):
    """The e4m3 value next to x (float64), ties to the even code, magnitudes over 448 to 448."""
    m = x.abs()
    e = torch.floor(torch.log2(m.clamp(min=2.0**-30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.sign(x) * (torch.round(m / step) * step).clamp(max=448)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        half, t = case["rot"] // 2, case["tokens"]
        axis = s["axis_of"] or [0] * half
        pos = s["positions"].view(-1, t).cpu()
        cs = s["cos_sin"].double()
        c = torch.stack([cs[pos[a].long().to(DEV), i] for i, a in enumerate(axis)], 1)
        n = torch.stack([cs[pos[a].long().to(DEV), half + i] for i, a in enumerate(axis)], 1)
        out = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.double()
            if w is not None:
                x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + 1e-6)
            z = torch.complex(c, n)[:, None]
            y = x.clone()
            if case["pairs"]:
                turned = torch.complex(x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]) * z
                y[..., 0 : 2 * half : 2], y[..., 1 : 2 * half : 2] = turned.real, turned.imag
            else:
                turned = torch.complex(x[..., :half], x[..., half : 2 * half]) * z
                y[..., :half], y[..., half : 2 * half] = turned.real, turned.imag
            out.append(y)
        return tuple(out)
    if op in ("append", "read"):
        p, loc = case["page"], s["loc"].long()
        hnd = case["layout"] == "HND"
        heads = torch.arange(case["kv_heads"], device=DEV)[None]
        page, slot = (loc // p)[:, None], (loc % p)[:, None]
        where = (page, heads, slot) if hnd else (page, slot, heads)
        if op == "read":
            return tuple(pool.to(torch.float64)[where] * scale.double()[where][..., None]
                         for pool, scale in zip(s["pools"], s["scales"]))
        pools, scales = [], []
        for new, pool, scale in zip((s["k_new"], s["v_new"]), s["pools"], s["scales"]):
            x = new.double()
            top = x.abs().amax(-1)
            ratio = top.clamp(min=1e-300) / 448
            unit = torch.exp2(torch.round(torch.log2(ratio)))
            unit = torch.where(top > 0, torch.where(unit >= ratio, unit, 2 * unit), 1.0)
            pool, scale = pool.to(torch.float64), scale.double()
            pool[where] = _nearest_e4m3(x / unit[..., None])
            scale[where] = unit
            pools.append(pool)
            scales.append(scale)
        return (*pools, *scales)
    n, kv = _tree_lens(case)
    p, hnd, grp = case["page"], case["layout"] == "HND", case["heads"] // case["kv_heads"]
    bits = s["mask"].cpu().tolist()
    out, row = [], 0
    for b, (m, length) in enumerate(zip(n, kv)):
        used = s["table"][b, : -(-length // p)].long()
        k, v = (x.view(torch.uint8)[used].view(E4M3) if x.dtype == E4M3 else x[used] for x in s["pools"])
        k, v = (x.to(torch.float64).permute(1, 0, 2, 3) if hnd else x.to(torch.float64).permute(2, 0, 1, 3) for x in (k, v))
        k, v = (x.reshape(case["kv_heads"], -1, case["dim"])[:, :length] for x in (k, v))
        see = torch.zeros((m, length), dtype=torch.bool)
        ctx = length - m
        for i in range(m):
            far = 0 if case["window"] < 0 else max(0, int(s["positions"][row + i]) - case["window"])
            see[i, far:ctx] = True
            for j in range(m):
                see[i, ctx + j] = bits[row + i][j // 32] >> (j % 32) & 1 == 1
        see = see.to(DEV)
        q = s["q"][row : row + m].double().permute(1, 0, 2).reshape(case["kv_heads"], grp * m, -1)
        x = torch.matmul(q, k.transpose(1, 2)).view(case["heads"], m, length) * s["bmm1"]
        x = torch.where(see, x, -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        e = torch.exp(x - top)
        den = e.sum(-1, keepdim=True)
        if s["sinks"] is not None:
            den = den + torch.exp(s["sinks"].double().view(-1, 1, 1) - top)
        o = torch.matmul(e.view(case["kv_heads"], grp * m, length), v).view(case["heads"], m, -1) / den * s["bmm2"]
        out.append(o.permute(1, 0, 2))
        row += m
    return torch.cat(out)
