"""The stream that a call is given: an integer handle, 0 among them, means that very stream."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def caches():
    k, v = (torch.zeros((4, 2, 16, 128), dtype=F8, device=DEV) for _ in "kv")
    ks, vs = (torch.ones((4, 2, 16), device=DEV) for _ in "kv")
    return (k, v), (ks, vs)


def calls(b2pa, stream):
    """Each call around the attention with an input that sets a bit of the device error word of its stream."""
    pools, scales = caches()
    rows = torch.ones((1, 2, 128), dtype=BF, device=DEV)
    out = torch.tensor([-1], dtype=torch.int32, device=DEV)
    q = torch.ones((1, 4, 128), dtype=BF, device=DEV)
    one, cum = torch.ones(1, dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    table = torch.full((1, 1), 99, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    yield b2pa.DEV_BAD_SLOT, lambda: b2pa.append_kv_scaled(rows, rows, pools, scales, out, stream=stream)
    yield b2pa.DEV_BAD_SLOT, lambda: b2pa.read_kv_scaled(pools, scales, out, stream=stream)
    yield b2pa.DEV_BAD_POSITION, lambda: b2pa.qk_norm_rope(q, rows, torch.ones((8, 128), device=DEV), out, stream=stream)
    yield b2pa.DEV_BAD_PAGE, lambda: b2pa.tree_attention(q, pools, table, one, one.view(1, 1), 1, 1, 1.0, 1.0, cum,
                                                         stream=stream)


@pytest.mark.parametrize("which", ["default", "other"])
@pytest.mark.parametrize("form", ["handle", "stream"])
@pytest.mark.parametrize("current", [False, True])
def test_the_call_runs_on_the_stream_it_names(cuda_lib, which, form, current):
    s = torch.cuda.default_stream() if which == "default" else torch.cuda.Stream()
    assert (s.cuda_stream == 0) == (which == "default")
    # (made while another stream is current, or while this one is)
    with torch.cuda.stream(s if current else torch.cuda.Stream()):
        for bit, call in calls(cuda_lib, s.cuda_stream if form == "handle" else s):
            call()
            assert cuda_lib.device_status(s.cuda_stream) == bit
            assert cuda_lib.device_status(s.cuda_stream) == 0


def test_handle_zero_is_ordered_with_the_default_stream(cuda_lib):
    """Inputs written late on the default stream, and the result read there, with no other synchronisation."""
    q = torch.zeros((64, 4, 128), dtype=BF, device=DEV)
    k = torch.zeros((64, 2, 128), dtype=BF, device=DEV)
    cs = torch.cat([torch.ones((64, 64)), torch.zeros((64, 64))], 1).to(DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    cuda_lib.qk_norm_rope(q, k, cs, pos, stream=0)
    torch.cuda.synchronize()
    for i in range(1, 6):
        torch.cuda._sleep(20_000_000)
        q.fill_(float(i))
        k.fill_(float(-i))
        a, b = cuda_lib.qk_norm_rope(q, k, cs, pos, stream=0)
        assert (a == i).all() and (b == -i).all()
