"""What the page ledger, page copies and compaction refuse on the host, before any CUDA call: the C entry points with
descriptors that point nowhere, and the Python functions with tensors that are not on a GPU."""
import ctypes

import pytest
import torch

from test_ops_refusals import BF, F8, F32, I32, INVALID, OK, UNSUPPORTED, fake, ref
from test_ops_refusals import lib  # noqa: F401

M = 1 << 20


def copy(lib, **change):
    a = dict(k=fake([5, 2, 16, 64], BF), v=fake([5, 2, 16, 64], BF), ks=None, vs=None, src=fake([3], I32),
             dst=fake([3], I32, base=2 * M), layout=0)
    a.update(change)
    return lib.b2pa_copy_pages(*(ref(a[x]) for x in ("k", "v", "ks", "vs", "src", "dst")), a["layout"], None)


@pytest.mark.parametrize("change,status", [
    (dict(k=None), INVALID),
    (dict(k=fake([5, 2, 16, 64], F32)), INVALID),
    (dict(v=fake([5, 2, 16, 64], F8)), INVALID),
    (dict(v=fake([6, 2, 16, 64], BF)), INVALID),
    (dict(k=fake([5, 2, 16, 64], BF, [0, 1024, 64, 1])), INVALID),         # one page five times
    (dict(v=fake([5, 2, 16, 64], BF, [2048, 1024, 32, 1])), INVALID),      # rows that overlap
    (dict(v=fake([5, 2, 16, 64], BF, [2048, 512, 64, 1])), INVALID),       # heads that overlap
    (dict(k=fake([5, 2, 16, 64], BF, [-2048, 1024, 64, 1])), INVALID),
    (dict(layout=3), INVALID),
    (dict(ks=fake([5, 2, 16], F32)), INVALID),                             # K's scales alone
    (dict(ks=fake([5, 2, 16], F32), vs=fake([5, 16, 2], F32)), INVALID),
    (dict(ks=fake([5, 2, 16], F32, [0, 16, 1]), vs=fake([5, 2, 16], F32)), INVALID),
    (dict(src=None), INVALID),
    (dict(src=fake([4], I32)), INVALID),
    (dict(src=fake([3], F32)), INVALID),
    (dict(dst=fake([3], I32, [2])), INVALID),
    (dict(dst=fake([3], I32, base=0)), INVALID),
    (dict(dst=fake([3, 1], I32)), INVALID),
])
def test_copy_pages(lib, change, status):  # noqa: F811
    assert copy(lib, **change) == status
    assert lib.b2pa_last_error_message()


def test_copy_of_no_pages(lib):  # noqa: F811
    assert copy(lib, src=fake([0], I32, base=0), dst=fake([0], I32, base=0)) == OK


def compact(lib, **change):
    a = dict(k=fake([5, 2, 16, 64], F8), v=fake([5, 2, 16, 64], F8), ks=None, vs=None, table=fake([3, 4], I32),
             seq=fake([3], I32), cum=fake([4], I32), acc=fake([3, 7], I32), counts=fake([3], I32, base=3 * M),
             out=fake([3], I32, base=2 * M), layout=1)
    a.update(change)
    return lib.b2pa_compact_kv(*(ref(a[x]) for x in ("k", "v", "ks", "vs", "table", "seq", "cum", "acc", "counts", "out")),
                               a["layout"], None)


@pytest.mark.parametrize("change", [
    dict(k=None), dict(k=fake([5, 2, 16, 64], BF)), dict(table=fake([2, 4], I32)), dict(table=fake([3, 4], I32, [4, 2])),
    dict(table=None), dict(table=fake([3], I32)), dict(seq=fake([3], F32)), dict(seq=None), dict(cum=fake([3], I32)),
    dict(cum=None), dict(acc=fake([2, 7], I32)), dict(acc=fake([3, 7], F32)), dict(acc=fake([3, 7], I32, [1, 3])),
    dict(acc=fake([3, 7], I32, base=0)), dict(counts=fake([4], I32)), dict(counts=None), dict(out=None),
    dict(out=fake([2], I32, base=2 * M)), dict(out=fake([3], I32, [2], base=2 * M)),
    dict(out=fake([3], I32)),                        # new_lens is seq_lens
    dict(out=fake([3], I32, base=3 * M)),            # new_lens is counts
    dict(vs=fake([5, 2, 16], F32)), dict(layout=-1),
])
def test_compact(lib, change):  # noqa: F811
    assert compact(lib, **change) == INVALID
    assert lib.b2pa_last_error_message()


@pytest.mark.parametrize("change", [
    dict(out=fake([3], I32, base=M + 4)),                   # in the tables, the lengths, the nodes
    dict(counts=fake([3], I32, base=2 * M - 8)),            # the last one is new_lens[0]
    dict(acc=fake([3, 7], I32, [32, 1], base=2 * M - 256)),
])
def test_compact_over_inputs(lib, change):  # noqa: F811
    assert compact(lib, **change) == INVALID
    assert lib.b2pa_last_error_message()


def test_compact_of_no_requests(lib):  # noqa: F811
    none = fake([0], I32, base=0)
    assert compact(lib, table=fake([0, 4], I32, base=0), seq=none, cum=fake([1], I32), acc=fake([0, 7], I32, base=0),
                   counts=none, out=none) == OK


def ledger(lib, call, **change):
    a = dict(table=fake([6, 9], I32), seq=fake([6], I32), refs=fake([50], I32), rows=fake([3], I32),
             more=fake([3], I32, base=2 * M), page=16, src=fake([3], I32, base=3 * M), dst=fake([3], I32, base=4 * M))
    a.update(change)
    d = [ref(a[x]) for x in ("table", "seq", "refs")]
    if call == "free":
        return lib.b2pa_free_pages(*d, ref(a["rows"]), a["page"], None)
    if call == "grow":
        return lib.b2pa_grow_pages(*d, ref(a["rows"]), ref(a["more"]), a["page"], None)
    return lib.b2pa_fork_pages(*d, ref(a["more"]), ref(a["rows"]), a["page"], ref(a["src"]), ref(a["dst"]), None)


@pytest.mark.parametrize("call", ["free", "fork", "grow"])
@pytest.mark.parametrize("change,status", [
    (dict(table=None), INVALID),
    (dict(table=fake([5, 9], I32)), INVALID),
    (dict(table=fake([6, 9], F32)), INVALID),
    (dict(table=fake([6, 9], I32, [1, 6])), INVALID),
    (dict(table=fake([6, 9], I32, [8, 1])), INVALID),                      # rows that overlap
    (dict(table=fake([6, 9], I32, base=0)), INVALID),
    (dict(table=fake([6, 1 << 30], I32)), INVALID),
    (dict(seq=fake([6], F32)), INVALID),
    (dict(seq=None), INVALID),
    (dict(refs=fake([50], I32, [2])), INVALID),
    (dict(refs=fake([1 << 30], I32)), INVALID),
    (dict(refs=fake([50, 1], I32)), INVALID),
    (dict(rows=None), INVALID),
    (dict(rows=fake([3], F32)), INVALID),
    (dict(page=0), INVALID),
    (dict(page=-16), INVALID),
    (dict(rows=fake([4097], I32)), UNSUPPORTED),
])
def test_ledger(lib, call, change, status):  # noqa: F811
    assert ledger(lib, call, **change) == status
    assert lib.b2pa_last_error_message()


@pytest.mark.parametrize("call,change", [
    ("fork", dict(more=fake([2], I32))), ("fork", dict(more=None)), ("fork", dict(src=None)),
    ("fork", dict(src=fake([4], I32, base=3 * M))), ("fork", dict(dst=fake([3], F32))),
    ("fork", dict(dst=fake([3], I32, base=3 * M))), ("grow", dict(more=fake([2], I32))), ("grow", dict(more=None)),
])
def test_ledger_arguments(lib, call, change):  # noqa: F811
    assert ledger(lib, call, **change) == INVALID
    assert lib.b2pa_last_error_message()


@pytest.mark.parametrize("call", ["free", "fork", "grow"])
def test_ledger_of_no_requests(lib, call):  # noqa: F811
    none = fake([0], I32, base=0)
    assert ledger(lib, call, rows=none, more=none, src=none, dst=none) == OK


APART = dict(table=fake([6, 9], I32, [12, 1], base=5 * M), seq=fake([6], I32, base=6 * M), refs=fake([50], I32, base=7 * M),
             rows=fake([3], I32, base=8 * M))
AT = dict(table=5 * M, seq=6 * M, refs=7 * M, rows=8 * M, more=2 * M, src=3 * M, dst=4 * M)
PAIRS = [("free", a, b) for a, b in (("table", "seq"), ("table", "refs"), ("table", "rows"), ("seq", "refs"), ("seq", "rows"),
                                     ("refs", "rows"))]
PAIRS += [(call, a, "more") for call in ("fork", "grow") for a in ("table", "seq", "refs")]
PAIRS += [("fork", a, b) for b in ("src", "dst") for a in ("table", "seq", "refs")] + [("fork", "src", "dst")]


def place(name, base):
    return fake([6, 9], I32, [12, 1], base=base) if name == "table" else fake(
        [dict(seq=6, refs=50).get(name, 3)], I32, base=base)


@pytest.mark.parametrize("call,a,b", PAIRS)
def test_ledger_over_itself_or_its_arguments(lib, call, a, b):  # noqa: F811
    """A tensor that is written over any that is read or written: by its first and by its last element."""
    last = {"table": 4 * (5 * 12 + 8), "seq": 4 * 5, "refs": 4 * 49}
    for base in (AT[a], AT[a] + last.get(a, 8), AT[a] - last.get(b, 8)):
        assert ledger(lib, call, **{**APART, b: place(b, base)}) == INVALID
        assert b"overlap" in lib.b2pa_last_error_message()


def test_ledger_arguments_that_reach_into_a_row(lib):  # noqa: F811
    """(Between a table's rows there may be room, in which a tensor may lie whole.)"""
    for at in (12 + 8, 12 + 10, 2 * 12 - 1, 5 * 12 + 8, -2):
        assert ledger(lib, "grow", **{**APART, "more": fake([3], I32, base=5 * M + 4 * at)}) == INVALID
        assert b"overlap" in lib.b2pa_last_error_message()


def test_python_functions_want_cuda_tensors(lib):  # noqa: F811
    import paged_kv_prefill_gb300 as b2pa

    pools = (torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16),) * 2
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 4), dtype=torch.int32)
    for call in (lambda: b2pa.copy_pages(pools, i, i), lambda: b2pa.compact_kv(pools, t, i, torch.zeros(3).int(), t, i),
                 lambda: b2pa.free_pages(t, i, i, i, 16), lambda: b2pa.fork_pages(t, i, i, i, i, 16),
                 lambda: b2pa.grow_pages(t, i, i, i, i, 16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="kv_scales"):
        b2pa.copy_pages(pools, i, i, kv_scales=i)
    with pytest.raises(KeyError):
        b2pa.copy_pages(pools, i, i, kv_layout="NDH")
