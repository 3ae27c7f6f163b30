"""Keys that are not finite, and values behind weights that underflow, in attention whose rows are put together from
parts: a row that sees such a key is NaN, whatever the parts are; the others are as the formula says."""
import math

import pytest
import torch

from test_gpu_prefix import F8, Batch
from test_gpu_tree import Batch as Trees

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CFG = {"bf16": dict(H=8, Hkv=2, D=128), "d64": dict(H=8, Hkv=2, D=64), "e4m3": dict(H=8, Hkv=2, D=128, cache="e4m3"),
       "heads_16": dict(H=32, Hkv=2, D=128), "heads_16_e4m3": dict(H=32, Hkv=2, D=128, cache="e4m3"),
       "heads_20": dict(H=40, Hkv=2, D=128)}


def nan(x):
    (x.view(torch.uint8) if x.dtype == F8 else x).fill_(0x7F if x.dtype == F8 else math.nan)


def put(t, pool, table, key, d=slice(None)):
    """NaN in dims d of all heads of a key (HND pools)."""
    row = pool[int(table[key // t.P]), :, key % t.P]
    nan(row[:, d] if row.dtype != F8 else row.view(torch.uint8)[:, d].view(F8))


@pytest.fixture(params=["auto", "generic"])
def path(cuda_lib, request):
    cuda_lib.set_kernel_path(request.param)
    yield request.param
    cuda_lib.set_kernel_path("auto")


@pytest.mark.parametrize("cfg", CFG)
def test_own_keys(cuda_lib, path, cfg):
    """The only own key; the only one of 16, and of a tile; all of them; behind a finite prefix of many keys and of
    one, and behind none."""
    kvs = [1, 17, 40, 129, 33, 5, 1, 1, 9]
    t = Batch([5, 2], [300, 1], [1] * 9, kvs, P=16, seed=4, **CFG[cfg])
    hit = {0: [0], 1: [16], 3: [128], 4: list(range(33)), 6: [0], 7: [0]}
    for b, keys in hit.items():
        for key in keys:
            put(t, t.k, t.table[b], key)
    out = cuda_lib.prefix_attention(**t.dev())
    assert cuda_lib.device_status() == 0
    for b in range(9):
        assert torch.isnan(out[b]).all() if b in hit else True, b
    t.check(out, [b for b in range(9) if b not in hit])


@pytest.mark.parametrize("cfg", CFG)
def test_keys_of_later_tokens(cuda_lib, path, cfg):
    """A request's last key reaches its last row; its other rows are as without it."""
    t = Batch([3], [200], [3, 2, 40], [50, 2, 300], P=16, seed=4, **CFG[cfg])
    good = cuda_lib.prefix_attention(**t.dev())
    t.check(good)
    for b in range(3):
        put(t, t.k, t.table[b], t.kvs[b] - 1)
    out = cuda_lib.prefix_attention(**t.dev())
    for b in range(3):
        assert torch.isnan(out[t.cum[b + 1] - 1]).all(), b
        assert torch.equal(out[t.cum[b] : t.cum[b + 1] - 1], good[t.cum[b] : t.cum[b + 1] - 1]), b
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cfg", CFG)
@pytest.mark.parametrize("length", [1, 130, 1000])
def test_whole_prefixes(cuda_lib, path, cfg, length):
    t = Batch([3, 2], [length, 140], [1] * 5, [7, 30, 300, 9, 200], P=16, seed=4, **CFG[cfg])
    for key in range(length):
        put(t, t.k, t.ptable[0], key)
    out = cuda_lib.prefix_attention(**t.dev())
    assert torch.isnan(out[:3]).all()
    t.check(out, [3, 4])
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cfg", CFG)
@pytest.mark.parametrize("which", ["prefix", "own"])
def test_parts_cut_over_ctas(cuda_lib, cfg, which):
    """Every run of one to three tiles of a long row of them, so that some run is just what a CTA took."""
    long = 32 * 128
    t = Batch([3], [long if which == "prefix" else 100], [1] * 3, [long if which == "own" else 60, 9, 30], P=128, seed=4,
              **CFG[cfg])
    d = t.dev()
    pool = d["kv_cache"][0]
    table = t.ptable[0] if which == "prefix" else t.table[0]
    rows = 3 if which == "prefix" else 1
    for count in (1, 2, 3):
        for first in range(0, 32 - count + 1):
            pages = [int(x) for x in table[first : first + count]]
            for pg in pages:
                nan(pool[pg])
            out = cuda_lib.prefix_attention(**d)
            assert torch.isnan(out[:rows]).all(), (count, first)
            for pg in pages:
                pool[pg].view(torch.uint8).copy_(t.k[pg].view(torch.uint8))
    t.check(cuda_lib.prefix_attention(**d))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cfg", CFG)
def test_values_behind_weights_that_underflow(cuda_lib, path, cfg):
    """Scores 0 but for one own key's, 181 above: the others' weights are 0 in 32 bits, and NaN among their values
    is NaN all the same."""
    t = Batch([2, 1], [300, 40], [1] * 3, [40, 17, 5], P=16, seed=4, **CFG[cfg])
    big = 4 * 50 if t.cache == "e4m3" else 4.0
    t.q.fill_(4.0 * math.sqrt(128 / t.D))
    t.k.copy_(torch.zeros(t.k.shape))
    for b, key in ((0, 39), (1, 16), (2, 4)):
        t.k[int(t.table[b, key // t.P]), :, key % t.P] = torch.full((t.Hkv, t.D), big).to(t.k.dtype)
    put(t, t.v, t.ptable[0], 7, slice(3, 4))   # both of the first group
    put(t, t.v, t.table[2], 1, slice(5, 6))    # the last request
    out = cuda_lib.prefix_attention(**t.dev())
    assert torch.isnan(out[:2, :, 3]).all() and torch.isnan(out[2, :, 5]).all()
    ok = torch.ones(t.D, dtype=torch.bool, device=DEV)
    ok[3] = False
    assert torch.isfinite(out[:2][..., ok]).all()
    put(t, t.v, t.table[0], 2, slice(9, 10))   # in another warp's keys than the large one
    out = cuda_lib.prefix_attention(**t.dev())
    assert torch.isnan(out[0, :, 9]).all() and torch.isfinite(out[1, :, 9]).all()
    assert cuda_lib.device_status() == 0


TREES = {"bf16": dict(H=8, Hkv=2, D=128), "d64": dict(H=8, Hkv=2, D=64), "e4m3": dict(H=8, Hkv=2, D=128, cache="e4m3")}


@pytest.mark.parametrize("cfg", TREES)
@pytest.mark.parametrize("n", [5, 40])
@pytest.mark.parametrize("tiles", [16, 64])
def test_trees_cut_over_ctas(cuda_lib, cfg, n, tiles):
    """The same for the context of a drafted tree."""
    t = Trees([n], [tiles * 128 + n], P=128, seed=4, **TREES[cfg])
    d = t.dev()
    pool = d["kv_cache"][0]
    for count in (1, 2, 3):
        for first in range(0, tiles - count + 1):
            pages = [int(x) for x in t.table[0, first : first + count]]
            for pg in pages:
                nan(pool[pg])
            out = cuda_lib.tree_attention(**d)
            assert torch.isnan(out).all(), (count, first)
            for pg in pages:
                pool[pg].view(torch.uint8).copy_(t.k[pg].view(torch.uint8))
    t.check(cuda_lib.tree_attention(**d))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("cfg", TREES)
def test_tree_values_behind_weights_that_underflow(cuda_lib, cfg):
    """Scores 0 in the context, 181 and more in the nodes' own keys; NaN among the context's values."""
    n, tiles = 5, 32
    t = Trees([n], [tiles * 128 + n], P=128, seed=4, **TREES[cfg])
    t.q.fill_(4.0 * math.sqrt(128 / t.D))
    t.k.copy_(torch.zeros(t.k.shape))
    for key in range(tiles * 128, tiles * 128 + n):
        t.k[int(t.table[0, key // 128]), :, key % 128] = torch.full(
            (t.Hkv, t.D), 200.0 if t.cache == "e4m3" else 4.0).to(t.k.dtype)
    for tile in (0, 9, 31):
        put(t, t.v, t.table[0], tile * 128 + 3, slice(tile, tile + 1))
    out = cuda_lib.tree_attention(**t.dev())
    assert torch.isnan(out[..., [0, 9, 31]]).all()
    assert torch.isfinite(out[..., 1:9]).all()
    assert cuda_lib.device_status() == 0
