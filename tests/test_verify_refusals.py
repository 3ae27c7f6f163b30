"""What the verification of drafted trees refuses on the host, before any CUDA call."""
import pytest
import torch

from test_ops_refusals import BF, F32, I32, INVALID, OK, UNSUPPORTED, fake, ref
from test_ops_refusals import lib  # noqa: F401

M = 1 << 20


def verify(lib, **change):
    a = dict(target=fake([9, 50], F32), draft=None, tokens=fake([9], I32), parents=fake([9], I32),
             uniforms=fake([9], F32), last=fake([2], F32), cum=fake([3], I32), max_q=7, acc=fake([2, 7], I32, base=2 * M),
             counts=fake([2], I32, base=3 * M), next=fake([2], I32, base=4 * M))
    a.update(change)
    first = [ref(a[x]) for x in ("target", "draft", "tokens", "parents", "uniforms", "last", "cum")]
    return lib.b2pa_verify_trees(*first, a["max_q"], *(ref(a[x]) for x in ("acc", "counts", "next")), None)


@pytest.mark.parametrize("change,status", [
    (dict(target=None), INVALID),
    (dict(target=fake([9, 50], BF)), INVALID),
    (dict(target=fake([9], F32)), INVALID),
    (dict(target=fake([9, 0], F32)), INVALID),
    (dict(target=fake([9, 50], F32, [1, 9])), INVALID),
    (dict(target=fake([9, 50], F32, [-50, 1])), INVALID),
    (dict(target=fake([9, 50], F32, base=0)), INVALID),
    (dict(target=fake([9, 50], F32, base=M + 2)), INVALID),
    (dict(target=fake([9, 1 << 30], F32)), INVALID),
    (dict(draft=fake([9, 49], F32)), INVALID),
    (dict(draft=fake([8, 50], F32)), INVALID),
    (dict(draft=fake([9, 50], BF)), INVALID),
    (dict(tokens=fake([8], I32)), INVALID),
    (dict(tokens=fake([9], F32)), INVALID),
    (dict(tokens=None), INVALID),
    (dict(parents=fake([9], I32, [2])), INVALID),
    (dict(parents=None), INVALID),
    (dict(uniforms=fake([9], I32)), INVALID),
    (dict(uniforms=fake([9, 1], F32)), INVALID),
    (dict(uniforms=None), INVALID),
    (dict(last=fake([3], F32)), INVALID),
    (dict(last=None), INVALID),
    (dict(cum=fake([2], I32)), INVALID),
    (dict(cum=None), INVALID),
    (dict(max_q=-1), INVALID),
    (dict(max_q=8), INVALID),                                              # accepted is narrower
    (dict(max_q=4097, acc=fake([2, 5000], I32)), UNSUPPORTED),
    (dict(acc=None), INVALID),
    (dict(acc=fake([2, 7], F32)), INVALID),
    (dict(acc=fake([3, 7], I32)), INVALID),
    (dict(acc=fake([2, 7], I32, [1, 2])), INVALID),
    (dict(acc=fake([2, 7], I32, [6, 1])), INVALID),
    (dict(acc=fake([2, 7], I32, base=3 * M)), INVALID),                    # in the place of counts
    (dict(counts=fake([2], F32)), INVALID),
    (dict(counts=None), INVALID),
    (dict(next=fake([3], I32)), INVALID),
    (dict(next=fake([2], I32, base=3 * M)), INVALID),
])
def test_verify(lib, change, status):  # noqa: F811
    assert verify(lib, **change) == status
    assert lib.b2pa_last_error_message()


@pytest.mark.parametrize("change", [
    dict(acc=fake([2, 7], I32)),                                           # begins where inputs do
    dict(target=fake([9, 50], F32, base=3 * M - 1796)),                    # its last value is counts[0]
    dict(draft=fake([9, 50], F32, [64, 1], base=4 * M - 400)),             # next_tokens in its first row
    dict(parents=fake([9], I32, base=2 * M + 52)),                         # behind accepted's first row
    dict(cum=fake([3], I32, base=3 * M + 4)),
    dict(counts=fake([2], I32, base=2 * M + 32)),                          # in accepted's rows
    dict(next=fake([2], I32, base=3 * M + 4)),
])
def test_outputs_over_tensors(lib, change):  # noqa: F811
    """A request's thread blocks each read its nodes: what one writes must not be what another reads."""
    assert verify(lib, **change) == INVALID
    assert lib.b2pa_last_error_message()


def test_no_requests(lib):  # noqa: F811
    z = dict(tokens=fake([0], I32, base=0), parents=fake([0], I32, base=0), uniforms=fake([0], F32, base=0))
    assert verify(lib, target=fake([0, 50], F32, base=0), last=fake([0], F32, base=0), cum=fake([1], I32),
                  acc=fake([0, 7], I32, base=0), counts=fake([0], I32, base=0), next=fake([0], I32, base=0), **z) == OK


def test_python_function_wants_cuda_tensors(lib):  # noqa: F811
    import paged_kv_prefill_gb300 as b2pa

    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        b2pa.verify_trees(torch.ones((2, 4)), i, i, torch.rand(2), torch.rand(1), 2, i)
