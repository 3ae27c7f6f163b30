"""The e4m3 cache with one scale per row (b2pa_append_kv_scaled,
b2pa_read_kv_scaled) on the GPU, bit for bit against the definition in fp64."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def nearest_e4m3(x):
    """The e4m3 value next to x (float64), ties to the even code, saturating."""
    m = x.abs().clamp(max=1e30)
    _, e = torch.frexp(m)  # m = f 2^e, 0.5 <= f < 1
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.copysign((torch.round(m / step) * step).clamp(max=448.0), x)


def definition(x):
    """(values of the codes in fp64, scales) of bf16 rows."""
    x = x.double()
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    e = torch.full(top.shape, -126, dtype=torch.int32)
    for n in range(-126, 121):  # the smallest that fits
        e = torch.where(top > 448 * 2.0 ** n, n + 1, e)
    scale = torch.where(top == 0, 1.0, torch.exp2(e.double()))
    return torch.where(torch.isnan(x), x, nearest_e4m3(x / scale[..., None])), scale


def pools(layout, N, P, H, D, g):
    shape = (N, H, P, D) if layout == "HND" else (N, P, H, D)
    return ([torch.randint(0, 120, shape, generator=g, dtype=torch.uint8).view(F8) for _ in "kv"],
            [torch.exp2(torch.randint(-9, 9, shape[:3], generator=g).float()) for _ in "kv"])


def place(layout, pool, loc, P):
    """View of [N, P, Hkv, ..] and the (page, slot) of each token."""
    return (pool.transpose(1, 2) if layout == "HND" else pool), loc.long() // P, loc.long() % P


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=1e9), torch.nan_to_num(b.double(), nan=1e9))


CASES = [
    # layout, T, N, P, Hkv, D
    ("HND", 1, 2, 1, 1, 8),
    ("NHD", 33, 4, 16, 8, 128),
    ("HND", 777, 64, 32, 8, 128),
    ("NHD", 3001, 60, 64, 3, 64),
    ("HND", 2000, 90, 24, 4, 80),
    ("NHD", 5000, 170, 32, 2, 256),
    ("HND", 6000, 400, 16, 8, 72),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_write_and_read_back(cuda_lib, case):
    layout, T, N, P, H, D = case
    g = torch.Generator().manual_seed(11 + CASES.index(case))
    pool, scale = pools(layout, N, P, H, D, g)
    kv = torch.randn((T, 2, H, D), generator=g) * torch.exp2(torch.randint(-100, 100, (T, 2, H, 1), generator=g).float())
    kv = kv.to(BF)
    kv[T // 2] = 0
    loc = torch.randperm(N * P, generator=g)[:T].to(torch.int32)
    dp, ds = [x.to(DEV) for x in pool], [x.to(DEV) for x in scale]
    dkv = kv.to(DEV)
    cuda_lib.append_kv_scaled(dkv[:, 0], dkv[:, 1], dp, ds, loc.to(DEV), kv_layout=layout)
    assert cuda_lib.device_status() == 0
    for i in range(2):
        codes, unit = definition(kv[:, i])
        p, s = pool[i].double(), scale[i].double()
        v, page, slot = place(layout, p, loc, P)
        v[page, slot] = codes
        v, page, slot = place(layout, s, loc, P)
        v[page, slot] = unit
        assert same(dp[i].cpu(), p) and torch.equal(ds[i].cpu().double(), s)
    # rows back, in another order and some twice
    at = torch.randint(0, T, (T + 5,), generator=g)
    got = cuda_lib.read_kv_scaled(dp, ds, loc[at].to(DEV), kv_layout=layout)
    for i in range(2):
        codes, unit = definition(kv[:, i])
        back = codes * unit[..., None]
        assert same(back, back.to(BF))  # representable
        assert same(got[i].cpu(), back[at])
    # a second write of what was read back keeps every value
    rows = cuda_lib.read_kv_scaled(dp, ds, loc.to(DEV), kv_layout=layout)
    cuda_lib.append_kv_scaled(*rows, dp, ds, loc.to(DEV), kv_layout=layout)
    again = cuda_lib.read_kv_scaled(dp, ds, loc.to(DEV), kv_layout=layout)
    assert all(torch.equal(a, b) for a, b in zip(rows, again))


def test_special_values(cuda_lib):
    """Every bf16 magnitude as a row's largest value; ties; infinities, NaN, subnormals."""
    D, P = 8, 64
    tops = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(BF)
    T = tops.shape[0]
    g = torch.Generator().manual_seed(2)
    frac = torch.tensor([1.0, 0.75, -0.5, 0.3, 2.0 ** -9, -(2.0 ** -17), 2.0 ** -18, 0.0])
    x = (tops.double()[:, None, None] * frac.double()).to(BF)
    x[5::97, 0, 7] = float("inf")
    x[6::97, 0, 7] = -float("inf")
    x[7::97, 0, 6] = float("nan")
    loc = torch.randperm(T, generator=g).to(torch.int32)
    N = -(-T // P)
    pool, scale = pools("HND", N, P, 1, D, g)
    dp, ds = [v.to(DEV) for v in pool], [v.to(DEV) for v in scale]
    cuda_lib.append_kv_scaled(x.to(DEV), x.to(DEV), dp, ds, loc.to(DEV))
    codes, unit = definition(x)
    v, page, slot = place("HND", dp[1].cpu().double(), loc, P)
    assert same(v[page, slot], codes)
    v, page, slot = place("HND", ds[0].cpu().double(), loc, P)
    assert torch.equal(v[page, slot], unit)


def test_read_of_every_code_under_any_scale(cuda_lib):
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(F8).view(1, 1, 32, 8).contiguous()
    s = torch.tensor([1.0, 3.7, 1e-30, 2.0 ** -126, 1e36, -0.3, 0.0, float("nan")]).repeat(4).view(1, 1, 32)
    loc = torch.arange(32, dtype=torch.int32)
    k, v = cuda_lib.read_kv_scaled((codes.to(DEV), codes.to(DEV)), (s.to(DEV), s.to(DEV)), loc.to(DEV))
    ref = (codes.float() * s[..., None]).to(BF).view(32, 1, 8)
    assert same(k.cpu(), ref) and same(v.cpu(), ref)


def test_slots_outside_the_pool(cuda_lib):
    N, P, H, D, T = 6, 16, 2, 64, 50
    g = torch.Generator().manual_seed(4)
    pool, scale = pools("NHD", N, P, H, D, g)
    x = torch.randn((T, H, D), generator=g).to(BF)
    loc = torch.randperm(N * P, generator=g)[:T].to(torch.int32)
    bad = [3, 20, 49]
    loc[bad[0]], loc[bad[1]], loc[bad[2]] = -1, N * P, 2 ** 31 - 1
    ok = torch.ones(T, dtype=torch.bool)
    ok[bad] = False
    dp, ds = [v.to(DEV) for v in pool], [v.to(DEV) for v in scale]
    cuda_lib.append_kv_scaled(x.to(DEV), x.to(DEV), dp, ds, loc.to(DEV), kv_layout="NHD")
    assert cuda_lib.device_status() == cuda_lib.DEV_BAD_SLOT
    codes, unit = definition(x)
    p, s = pool[0].double(), scale[0].double()
    p[loc[ok].long() // P, loc[ok].long() % P] = codes[ok]
    s[loc[ok].long() // P, loc[ok].long() % P] = unit[ok]
    assert same(dp[0].cpu(), p) and torch.equal(ds[0].cpu().double(), s)
    k, _ = cuda_lib.read_kv_scaled(dp, ds, loc.to(DEV), kv_layout="NHD")
    assert cuda_lib.device_status() == cuda_lib.DEV_BAD_SLOT
    assert (k.cpu()[~ok] == 0).all() and same(k.cpu()[ok], (codes * unit[..., None])[ok])


def test_strided_pools_scales_and_outputs(cuda_lib):
    """One [N, 2, ...] cache, scales kept beside each other, outputs inside bf16 pools, K and V rows strided apart."""
    N, P, H, D, T = 5, 8, 4, 64, 37
    g = torch.Generator().manual_seed(6)
    cache = torch.zeros((N, 2, H, P, D), dtype=torch.uint8, device=DEV).view(F8)
    sc = torch.zeros((N, H, P, 2), device=DEV)
    k = torch.randn((H, T, D), generator=g).to(BF)
    v = torch.randn((T, H, D), generator=g).to(BF)
    loc = torch.randperm(N * P, generator=g)[:T].to(torch.int32).to(DEV)
    cuda_lib.append_kv_scaled(k.to(DEV).transpose(0, 1), v.to(DEV), cache, (sc[..., 0], sc[..., 1]), loc)
    out = torch.full((7, P, H, 2 * D), 9, dtype=BF, device=DEV)  # pages of bf16 K and V side by side
    rows = out.view(7 * P, H, 2 * D)
    cuda_lib.read_kv_scaled(cache, (sc[..., 0], sc[..., 1]), loc, k_out=rows[3 : 3 + T, :, :D],
                            v_out=rows[3 : 3 + T, :, D:])
    for got, x in ((rows[3 : 3 + T, :, :D], k.transpose(0, 1)), (rows[3 : 3 + T, :, D:], v)):
        codes, unit = definition(x)
        assert same(got.cpu(), codes * unit[..., None])
    assert (rows[:3] == 9).all() and (rows[3 + T :] == 9).all()


def test_offsets_past_32_bits(cuda_lib):
    """A pool of more than 2^32 bytes: slots at its end."""
    N, P, H, D = 70000, 64, 8, 128  # 4.6 GB of codes
    T = 100
    cache = torch.zeros((N, P, H, D), dtype=torch.uint8, device=DEV).view(F8)
    sc = torch.zeros((N, P, H), device=DEV)
    x = torch.randn((T, H, D)).to(BF)
    loc = (N * P - 1 - 3 * torch.arange(T)).to(torch.int32).to(DEV)
    cuda_lib.append_kv_scaled(x.to(DEV), x.to(DEV), (cache, cache), (sc, sc), loc, kv_layout="NHD")
    k, v = cuda_lib.read_kv_scaled((cache, cache), (sc, sc), loc, kv_layout="NHD")
    codes, unit = definition(x)
    assert same(k.cpu(), codes * unit[..., None]) and torch.equal(k, v)
    assert not cache.view(torch.uint8).view(N, -1)[: N - 8].any()


def test_no_tokens_streams_and_graphs(cuda_lib):
    N, P, H, D, T = 8, 16, 2, 128, 60
    g = torch.Generator().manual_seed(8)
    pool, scale = pools("HND", N, P, H, D, g)
    dp, ds = [v.to(DEV) for v in pool], [v.to(DEV) for v in scale]
    e = torch.empty((0, H, D), dtype=BF, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    cuda_lib.append_kv_scaled(e, e, dp, ds, none)
    assert cuda_lib.read_kv_scaled(dp, ds, none)[0].shape == (0, H, D)
    x, y = torch.randn((T, H, D), generator=g).to(BF), torch.randn((T, H, D), generator=g).to(BF)
    dx = x.to(DEV)
    loc = torch.randperm(N * P, generator=g)[:T].to(torch.int32).to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cuda_lib.append_kv_scaled(dx, dx, dp, ds, loc, stream=s)
    k, _ = cuda_lib.read_kv_scaled(dp, ds, loc, stream=s)
    s.synchronize()
    codes, unit = definition(x)
    assert same(k.cpu(), codes * unit[..., None])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.append_kv_scaled(dx, dx, dp, ds, loc)
        k, v = cuda_lib.read_kv_scaled(dp, ds, loc)
    dx.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    codes, unit = definition(y)
    assert same(k.cpu(), codes * unit[..., None]) and torch.equal(k, v)


def test_outputs_larger_than_the_memory(cuda_lib):
    """torch's own error for it, and the next call is fine."""
    pool = torch.zeros((1, 64, 1, 256), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scale = torch.ones((1, 64, 1), device=DEV)
    many = torch.zeros(8_000_000, dtype=torch.int32, device=DEV)  # 32 KiB of K and of V each
    with pytest.raises(torch.cuda.OutOfMemoryError):
        cuda_lib.read_kv_scaled((pool, pool), (scale, scale), many)
    k, v = cuda_lib.read_kv_scaled((pool, pool), (scale, scale), many[:3])
    assert (k == 0).all() and (v == 0).all() and cuda_lib.device_status() == 0
