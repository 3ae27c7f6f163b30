"""What the calls around the attention refuse on the host, before any CUDA
call: the C entry points with descriptors that point nowhere, and the Python
functions with tensors that are not on a GPU."""
import ctypes

import pytest
import torch

BF, F8, F32, I32 = 1, 2, 3, 4
OK, INVALID, UNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module")
def lib():
    from paged_kv_prefill_gb300 import build

    build.build()
    import paged_kv_prefill_gb300 as pkg

    return pkg.load()


def fake(shape, dtype, stride=None, base=1 << 20):
    import paged_kv_prefill_gb300 as pkg

    if stride is None:
        stride, n = [], 1
        for s in reversed(shape):
            stride.insert(0, n)
            n *= s
    return pkg.B2paTensor(base, dtype, len(shape), tuple(shape), tuple(stride))


def ref(d):
    return None if d is None else ctypes.byref(d)


# ---------------------------------------------------------------- norm and rotation

def rope(lib, **change):
    a = dict(q=fake([9, 4, 64], BF), k=fake([9, 2, 64], BF), cos_sin=fake([100, 32], F32), positions=fake([9], I32),
             q_weight=fake([64], BF), k_weight=None, eps=1e-6, axis_of=None, q_out=fake([9, 4, 64], BF),
             k_out=fake([9, 2, 64], BF))
    a.update(change)
    axes = None if a["axis_of"] is None else (ctypes.c_int32 * len(a["axis_of"]))(*a["axis_of"])
    return lib.b2pa_qk_norm_rope(ref(a["q"]), ref(a["k"]), ref(a["cos_sin"]), ref(a["positions"]), ref(a["q_weight"]),
                                 ref(a["k_weight"]), a["eps"], axes, 0, ref(a["q_out"]), ref(a["k_out"]), None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID),
    (dict(q=fake([9, 4, 64], F32)), INVALID),
    (dict(q=fake([9, 256], BF)), INVALID),
    (dict(k=fake([8, 2, 64], BF)), INVALID),                               # another T
    (dict(k=fake([9, 2, 32], BF)), INVALID),                               # another D
    (dict(q=fake([9, 4, 64], BF, [256, 64, 2])), INVALID),                 # head_dim not contiguous
    (dict(q=fake([9, 4, 64], BF, [260, 64, 1])), INVALID),                 # not in 16-byte steps
    (dict(q=fake([9, 4, 64], BF, base=(1 << 20) + 8)), INVALID),           # not 16-byte aligned
    (dict(q=fake([9, 4, 64], BF, base=0)), INVALID),
    (dict(q_out=fake([9, 4, 64], BF, [0, 64, 1])), INVALID),               # a broadcast output
    (dict(q_out=fake([9, 4, 64], BF, [256, 32, 1])), INVALID),             # its rows overlap
    (dict(k_out=fake([9, 4, 64], BF)), INVALID),
    (dict(k_out=None), INVALID),
    (dict(q_weight=fake([32], BF)), INVALID),
    (dict(q_weight=fake([64], I32)), INVALID),
    (dict(k_weight=fake([64], F32, base=(1 << 20) + 4)), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(cos_sin=fake([100, 33], F32)), INVALID),                         # odd
    (dict(cos_sin=fake([100, 66], F32)), INVALID),                         # wider than D
    (dict(cos_sin=fake([100, 32], BF)), INVALID),
    (dict(cos_sin=fake([0, 32], F32)), INVALID),
    (dict(positions=fake([8], I32)), INVALID),
    (dict(positions=fake([5, 9], I32), axis_of=[0] * 16), INVALID),        # five axes
    (dict(positions=fake([2, 9], I32)), INVALID),                          # whose frequency is whose?
    (dict(positions=fake([2, 9], I32), axis_of=[0] * 15 + [2]), INVALID),
    (dict(positions=fake([2, 9], I32), axis_of=[0] * 15 + [-1]), INVALID),
    (dict(positions=fake([9, 2], I32, [1, 9])), INVALID),
])
def test_rope(lib, change, status):
    assert rope(lib, **change) == status
    assert lib.b2pa_last_error_message()


def test_rope_outputs_in_place_of_other_rows(lib):
    """An output at an input's address is that input, by the same strides; two outputs are two."""
    M = 1 << 20
    x = dict(q=fake([9, 4, 64], BF, base=M), k=fake([9, 2, 64], BF, base=2 * M))
    q_out, k_out = fake([9, 4, 64], BF, base=3 * M), fake([9, 2, 64], BF, base=4 * M)
    for change in (dict(q_out=q_out, k_out=fake([9, 2, 64], BF, base=3 * M)),
                   dict(q_out=fake([9, 4, 64], BF, [64, 9 * 64, 1], base=M), k_out=k_out),
                   dict(q_out=q_out, k_out=fake([9, 2, 64], BF, [256, 64, 1], base=2 * M)),
                   dict(q_out=fake([9, 4, 64], BF, base=2 * M), k_out=k_out),
                   dict(q_out=q_out, k_out=fake([9, 2, 64], BF, base=M))):
        assert rope(lib, **x, **change) == INVALID
        assert b"in the place of" in lib.b2pa_last_error_message()


def test_rope_head_dims(lib):
    for D in (60, 264):
        x = dict(q=fake([9, 4, D], BF), k=fake([9, 2, D], BF), q_out=fake([9, 4, D], BF), k_out=fake([9, 2, D], BF))
        assert rope(lib, q_weight=None, **x) == UNSUPPORTED


def test_rope_of_no_tokens(lib):
    x = dict(q=fake([0, 4, 64], BF, base=0), k=fake([0, 2, 64], BF, base=0), q_out=fake([0, 4, 64], BF, base=0),
             k_out=fake([0, 2, 64], BF, base=0))
    assert rope(lib, positions=fake([0], I32, base=0), **x) == OK


# ---------------------------------------------------------------- scaled cache

def scaled(lib, write, **change):
    a = dict(rows=[fake([9, 2, 64], BF)] * 2, pools=[fake([5, 2, 16, 64], F8)] * 2, scales=[fake([5, 2, 16], F32)] * 2,
             loc=fake([9], I32), layout=0)
    a.update(change)
    r, p, s = a["rows"], a["pools"], a["scales"]
    if write:
        return lib.b2pa_append_kv_scaled(ref(r[0]), ref(r[1]), ref(p[0]), ref(p[1]), ref(s[0]), ref(s[1]), ref(a["loc"]),
                                         a["layout"], None)
    return lib.b2pa_read_kv_scaled(ref(p[0]), ref(p[1]), ref(s[0]), ref(s[1]), ref(a["loc"]), a["layout"], ref(r[0]),
                                   ref(r[1]), None)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("change,status", [
    (dict(pools=[fake([5, 2, 16, 64], BF)] * 2), INVALID),
    (dict(pools=[fake([5, 2, 16, 64], F8), fake([5, 2, 16, 32], F8)]), INVALID),
    (dict(pools=[fake([5, 2, 16, 64], F8), None]), INVALID),
    (dict(pools=[fake([5, 2, 16, 64], F8, base=(1 << 20) + 4)] * 2), INVALID),
    (dict(pools=[fake([5, 2, 16, 64], F8, [2052, 1024, 64, 1])] * 2), INVALID),
    (dict(layout=1), INVALID),                                             # Hkv is now 16
    (dict(layout=2), INVALID),
    (dict(scales=[fake([5, 2, 16], F32), fake([5, 16, 2], F32)]), INVALID),
    (dict(scales=[fake([5, 2, 16], BF)] * 2), INVALID),
    (dict(scales=[fake([5, 2, 16, 1], F32)] * 2), INVALID),
    (dict(scales=[fake([5, 2, 16], F32, base=(1 << 20) + 2)] * 2), INVALID),
    (dict(scales=[None, None]), INVALID),
    (dict(rows=[fake([9, 2, 64], BF), fake([8, 2, 64], BF)]), INVALID),
    (dict(rows=[fake([9, 2, 64], F32)] * 2), INVALID),
    (dict(rows=[fake([9, 2, 64], BF, [128, 64, 2])] * 2), INVALID),
    (dict(rows=[fake([9, 2, 64], BF, base=0)] * 2), INVALID),
    (dict(loc=fake([9, 1], I32)), INVALID),
    (dict(loc=fake([9], F32)), INVALID),
    (dict(loc=fake([9], I32, [2])), INVALID),
    (dict(loc=None), INVALID),
    (dict(rows=[fake([9, 2, 60], BF, [128, 64, 1])] * 2, pools=[fake([5, 2, 16, 60], F8, [2048, 1024, 64, 1])] * 2), UNSUPPORTED),
    (dict(rows=[fake([9, 2, 264], BF)] * 2, pools=[fake([5, 2, 16, 264], F8)] * 2), UNSUPPORTED),
    (dict(pools=[fake([1 << 20, 2, 4096, 64], F8)] * 2, scales=[fake([1 << 20, 2, 4096], F32)] * 2), UNSUPPORTED),
])
def test_scaled(lib, write, change, status):
    assert scaled(lib, write, **change) == status
    assert lib.b2pa_last_error_message()


def test_scaled_writes_need_places_apart(lib):
    assert scaled(lib, True, scales=[fake([5, 2, 16], F32, [32, 16, 0])] * 2) == INVALID
    assert scaled(lib, True, pools=[fake([5, 2, 16, 64], F8, [0, 1024, 64, 1])] * 2) == INVALID
    assert scaled(lib, False, rows=[fake([9, 2, 64], BF, [0, 64, 1])] * 2) == INVALID


def test_scaled_read_into_one_buffer(lib):
    assert scaled(lib, False) == INVALID
    assert b"in the place of" in lib.b2pa_last_error_message()


def test_scaled_of_no_tokens(lib):
    none = dict(rows=[fake([0, 2, 64], BF, base=0)] * 2, loc=fake([0], I32, base=0))
    assert scaled(lib, True, **none) == OK and scaled(lib, False, **none) == OK


# ---------------------------------------------------------------- trees

def tree(lib, bytes_needed=True, **change):
    a = dict(q=fake([9, 4, 128], BF), k=fake([5, 2, 16, 128], BF), v=fake([5, 2, 16, 128], BF), bt=fake([3, 4], I32),
             seq=fake([3], I32), cum=fake([4], I32), mask=fake([9, 2], I32), pos=None, max_q=33, max_kv=64, bmm1=0.1,
             bmm2=1.0, window=-1, sinks=None, layout=0, out=fake([9, 4, 128], BF))
    a.update(change)
    need = ctypes.c_uint64(7)
    return lib.b2pa_tree_attention(ref(a["q"]), ref(a["k"]), ref(a["v"]), ref(a["bt"]), ref(a["seq"]), ref(a["cum"]),
                                   ref(a["mask"]), ref(a["pos"]), a["max_q"], a["max_kv"], a["bmm1"], a["bmm2"],
                                   a["window"], ref(a["sinks"]), a["layout"], ref(a["out"]), None, 0,
                                   ctypes.byref(need) if bytes_needed else None, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=fake([9, 3, 128], BF), out=fake([9, 3, 128], BF)), INVALID),   # not a multiple of the kv heads
    (dict(q=fake([9, 4, 64], BF), out=fake([9, 4, 64], BF)), INVALID),
    (dict(q=fake([9, 4, 128], F32)), INVALID),
    (dict(v=fake([5, 2, 16, 128], F8)), INVALID),
    (dict(bt=fake([2, 4], I32)), INVALID),
    (dict(bt=fake([3, 4], I32, [1, 3])), INVALID),
    (dict(seq=fake([3], F32)), INVALID),
    (dict(cum=fake([3], I32)), INVALID),
    (dict(cum=None), INVALID),
    (dict(mask=None), INVALID),
    (dict(mask=fake([9], I32)), INVALID),
    (dict(mask=fake([8, 2], I32)), INVALID),
    (dict(mask=fake([9, 1], I32)), INVALID),                               # 33 nodes need two words
    (dict(mask=fake([9, 2], F32)), INVALID),
    (dict(mask=fake([9, 2], I32, [1, 9])), INVALID),
    (dict(window=4), INVALID),                                             # a window needs positions
    (dict(window=4, pos=fake([8], I32)), INVALID),
    (dict(window=0, pos=fake([9], F32)), INVALID),
    (dict(max_q=-1), INVALID),
    (dict(max_kv=-1), INVALID),
    (dict(bmm1=0.0), INVALID),
    (dict(bmm1=float("inf")), INVALID),
    (dict(bmm2=float("nan")), INVALID),
    (dict(sinks=fake([3], F32)), INVALID),
    (dict(layout=3), INVALID),
    (dict(out=fake([9, 4, 128], BF, [0, 128, 1])), INVALID),
    (dict(out=fake([9, 4, 128], F32)), INVALID),
    (dict(out=None), INVALID),
    (dict(bytes_needed=False), INVALID),
    (dict(q=fake([9, 4, 512], BF), out=fake([9, 4, 512], BF), k=fake([5, 2, 16, 512], BF), v=fake([5, 2, 16, 512], BF)),
     UNSUPPORTED),
])
def test_tree(lib, change, status):
    assert tree(lib, **change) == status
    assert lib.b2pa_last_error_message()


def test_tree_in_place_and_too_long(lib):
    q = fake([9, 4, 128], BF, base=1 << 20)
    out = fake([9, 4, 128], BF, base=2 << 20)
    assert tree(lib, q=q, out=fake([9, 4, 128], BF, base=1 << 20)) == INVALID
    assert b"out must not be q" in lib.b2pa_last_error_message()
    assert tree(lib, q=q, out=out, max_kv=2**31 - 256) == UNSUPPORTED
    assert b"max_kv_len" in lib.b2pa_last_error_message()


@pytest.mark.parametrize("stride", [[128, 128, 1], [128, 1024, 1], [512, 64, 1], [256, 128, 1], [64, 1152, 1], [-512, 128, 1]])
def test_tree_rows_of_the_output_apart(lib, stride):
    assert tree(lib, out=fake([9, 4, 128], BF, stride, base=2 << 20)) == INVALID
    assert b"its rows overlap" in lib.b2pa_last_error_message()


def test_tree_of_nothing(lib):
    none = dict(q=fake([0, 4, 128], BF, base=0), out=fake([0, 4, 128], BF, base=0), mask=fake([0, 2], I32, base=0))
    assert tree(lib, **none) == OK
    assert tree(lib, bt=fake([0, 4], I32, base=0), seq=fake([0], I32, base=0), cum=fake([1], I32), **none) == OK


# ---------------------------------------------------------------- Python

def test_python_functions_want_cuda_tensors(lib):
    import paged_kv_prefill_gb300 as b2pa

    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    pool = torch.zeros((4, 2, 16, 64), dtype=torch.float8_e4m3fn)
    sc = torch.ones((4, 2, 16))
    with pytest.raises(ValueError, match="CUDA tensors"):
        b2pa.qk_norm_rope(x, x, torch.zeros((8, 64)), i)
    with pytest.raises(ValueError, match="CUDA tensors"):
        b2pa.append_kv_scaled(x, x, (pool, pool), (sc, sc), i)
    with pytest.raises(ValueError, match="CUDA tensors"):
        b2pa.read_kv_scaled((pool, pool), (sc, sc), i)
    with pytest.raises(ValueError, match="CUDA tensors"):
        b2pa.tree_attention(x, (pool, pool), i[:, None], i, i[:, None], 3, 8, 1.0, 1.0, i)
    with pytest.raises(TypeError, match="a pair"):
        b2pa.read_kv_scaled((pool, pool), sc, i)
    with pytest.raises(ValueError, match="one axis for each"):
        b2pa.qk_norm_rope(x, x, torch.zeros((8, 64)), i, axis_of=[0, 1])


def test_native_argument_types(lib):
    import paged_kv_prefill_gb300 as b2pa

    n = b2pa.native()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="arguments"):
        n.append_kv_scaled(0, x)
    with pytest.raises(TypeError, match="must be a tensor"):
        n.append_kv_scaled(0, None, x, x, x, x, x, x, 0)
