"""What the attention of shared prefixes refuses on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from test_ops_refusals import BF, F8, F32, I32, INVALID, OK, UNSUPPORTED, fake, ref
from test_ops_refusals import lib  # noqa: F401

M = 1 << 20


def prefix(lib, **change):
    a = dict(q=fake([9, 8, 64], BF), k=fake([20, 2, 16, 64], BF), v=fake([20, 2, 16, 64], BF), pt=fake([2, 7], I32),
             pl=fake([2], I32), cg=fake([3], I32), bt=fake([4, 6], I32), seq=fake([4], I32), cum=fake([5], I32),
             max_q=5, max_group=9, max_prefix=112, max_kv=96, bmm1=0.1, bmm2=1.0, sinks=None, layout=0,
             out=fake([9, 8, 64], BF, base=8 * M), need=True)
    a.update(change)
    need = ctypes.c_uint64(77)
    first = [ref(a[x]) for x in ("q", "k", "v", "pt", "pl", "cg", "bt", "seq", "cum")]
    st = lib.b2pa_prefix_attention(*first, a["max_q"], a["max_group"], a["max_prefix"], a["max_kv"], a["bmm1"], a["bmm2"],
                                   ref(a["sinks"]), a["layout"], ref(a["out"]), None, 0,
                                   ctypes.byref(need) if a["need"] else None, None)
    return st if st else need.value


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID),
    (dict(q=fake([9, 8, 64], F32)), INVALID),
    (dict(q=fake([9, 7, 64], BF)), INVALID),
    (dict(k=fake([20, 2, 16, 64], F8)), INVALID),
    (dict(v=fake([20, 2, 16, 128], BF)), INVALID),
    (dict(pt=None), INVALID),
    (dict(pt=fake([3, 7], I32)), INVALID),
    (dict(pt=fake([2, 7], F32)), INVALID),
    (dict(pt=fake([2, 7], I32, [1, 2])), INVALID),
    (dict(pt=fake([2, 7], I32, base=0)), INVALID),
    (dict(pl=None), INVALID),
    (dict(pl=fake([2], F32)), INVALID),
    (dict(pl=fake([2], I32, [3])), INVALID),
    (dict(cg=fake([2], I32)), INVALID),
    (dict(cg=None), INVALID),
    (dict(bt=fake([3, 6], I32)), INVALID),
    (dict(seq=fake([4], F32)), INVALID),
    (dict(cum=fake([4], I32)), INVALID),
    (dict(max_q=-1), INVALID),
    (dict(max_group=-1), INVALID),
    (dict(max_prefix=-1), INVALID),
    (dict(max_kv=-1), INVALID),
    (dict(max_prefix=2 ** 31 - 256), UNSUPPORTED),
    (dict(max_kv=2 ** 31 - 256), UNSUPPORTED),
    (dict(bmm1=0.0), INVALID),
    (dict(bmm1=float("inf")), INVALID),
    (dict(bmm2=float("nan")), INVALID),
    (dict(sinks=fake([7], F32)), INVALID),
    (dict(sinks=fake([8], BF)), INVALID),
    (dict(layout=2), INVALID),
    (dict(out=None), INVALID),
    (dict(out=fake([9, 8, 64], F32, base=8 * M)), INVALID),
    (dict(out=fake([9, 8, 64], BF, [0, 64, 1], base=8 * M)), INVALID),
    (dict(out=fake([9, 8, 64], BF)), INVALID),                             # out is q
    (dict(need=False), INVALID),
])
def test_prefix(lib, change, status):  # noqa: F811
    assert prefix(lib, **change) == status
    assert lib.b2pa_last_error_message()


def test_nothing_to_do(lib):  # noqa: F811
    none = fake([0], I32, base=0)
    assert prefix(lib, q=fake([0, 8, 64], BF, base=0), out=fake([0, 8, 64], BF, base=0)) == OK
    assert prefix(lib, q=fake([0, 8, 64], BF, base=0), out=fake([0, 8, 64], BF, base=0), bt=fake([0, 6], I32, base=0),
                  seq=none, cum=fake([1], I32), pt=fake([0, 7], I32, base=0), pl=none, cg=fake([1], I32)) == OK


def test_python_function(lib):  # noqa: F811
    import paged_kv_prefill_gb300 as b2pa

    pools = (torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16),) * 2
    q, i, t = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4)).int()
    with pytest.raises(ValueError, match="CUDA"):
        b2pa.prefix_attention(q, pools, t, i, i, t, i, 1, 64, 64, 0.1, 1.0, i)
    with pytest.raises(KeyError):
        b2pa.prefix_attention(q, pools, t, i, i, t, i, 1, 64, 64, 0.1, 1.0, i, kv_layout="DNH")
    with pytest.raises(ValueError, match="sinks"):
        b2pa.prefix_attention(q, pools, t, i, i, t, i, 1, 64, 64, 0.1, 1.0, i, sinks=[None, None])
