"""The run-time patterns' C ABI without a GPU: declared symbols, argument checks
on the host, scratch sizes."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 5
PTR = ctypes.c_void_p(4096)      # never dereferenced: the checks come first


@pytest.fixture(scope="module")
def dyn():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_dense_matrix_gb300.dynamic as m
    return m


def shape(dyn, **kw):
    s = dict(B=1, Tq=4, Tk=64, Hq=4, Hk=2, D=64, block=16, n=2, dtype=1, causal=1, scale=0.125)
    s.update(kw)
    return dyn._Shape(*(s[f] for f in ("B", "Tq", "Tk", "Hq", "Hk", "D", "block", "n", "dtype",
                                       "causal", "scale")), None)


def rows(dyn, data=4096, sb=8192, st=256, sh=64):
    return dyn._Rows(data, sb, st, sh)


def test_library_exports_every_declared_symbol(dyn):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "spmm_dynamic.h")).read(),
                 flags=re.S)
    names = sorted(set(re.findall(r"\b(spmm_[a-z_]+)\s*\(", src)))
    assert "spmm_blocks_attend" in names and "spmm_routes_sort" in names
    lib = ctypes.CDLL(os.path.join(ROOT, "sparse_dense_matrix_gb300", "libspmm.so"))
    assert not [n for n in names if not hasattr(lib, n)]


def test_public_names(dyn):
    import sparse_dense_matrix_gb300 as sdm
    for n in ("ExpertRoutes", "BlockSelection", "block_means", "select_blocks"):
        assert n in sdm.__all__ and getattr(sdm, n) is getattr(dyn, n)


def test_routes_refuse(dyn):
    L = dyn.lib
    assert L.spmm_routes_sort(PTR, 4, 2, 8, PTR, None, None, 0, None) == INVALID
    assert L.spmm_routes_sort(None, 4, 2, 8, PTR, PTR, None, 0, None) == INVALID
    assert L.spmm_routes_sort(PTR, -1, 2, 8, PTR, PTR, None, 0, None) == INVALID
    assert L.spmm_routes_sort(PTR, 4, 2, 2049, PTR, PTR, None, 0, None) == UNSUPPORTED
    assert L.spmm_routes_sort(PTR, 1 << 31, 2, 8, PTR, PTR, None, 0, None) == UNSUPPORTED
    need = L.spmm_routes_workspace(100000, 8, 64)
    assert need > 0 and L.spmm_routes_workspace(4, 2, 8) == 0
    assert L.spmm_routes_sort(PTR, 100000, 8, 64, PTR, PTR, None, 0, None) == INVALID
    assert L.spmm_routes_sort(PTR, 100000, 8, 64, PTR, PTR, PTR, need - 1, None) == INVALID
    assert L.spmm_routes_dispatch(3, PTR, 8, PTR, PTR, 4, 2, 8, 8, PTR, None) == INVALID
    assert L.spmm_routes_dispatch(0, PTR, -8, PTR, PTR, 4, 2, 8, 8, PTR, None) == INVALID
    assert L.spmm_routes_dispatch(0, None, 8, PTR, PTR, 4, 2, 8, 8, PTR, None) == INVALID
    assert L.spmm_routes_combine(0, PTR, None, None, PTR, 4, 2, 8, 8, PTR, None) == INVALID
    assert L.spmm_routes_combine(0, PTR, None, PTR, PTR, 4, 2, 8, 8, None, None) == INVALID
    assert L.spmm_routes_combine_backward(0, PTR, 8, PTR, None, PTR, PTR, 4, 2, 8, 8, None, None,
                                          None) == INVALID
    # nothing to do is no error, and needs no device
    assert L.spmm_routes_dispatch(0, None, 8, None, None, 0, 2, 8, 8, None, None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INVALID), (dict(Hq=5), INVALID), (dict(Hk=0), INVALID), (dict(n=0), INVALID),
    (dict(dtype=7), INVALID), (dict(block=48), UNSUPPORTED), (dict(D=63), UNSUPPORTED),
    (dict(D=264), UNSUPPORTED), (dict(Tk=1 << 27), UNSUPPORTED),
    (dict(Tq=1 << 20, Hq=4096), UNSUPPORTED)])
def test_blocks_refuse_shapes(dyn, bad, status):
    L, s, r = dyn.lib, shape(dyn, **bad), rows(dyn)
    assert L.spmm_blocks_means(s, r, -1, PTR, None) == status
    assert L.spmm_blocks_select(s, r, PTR, PTR, PTR, 1 << 40, None) == status
    assert L.spmm_blocks_check(s, PTR, PTR, None) == status
    assert L.spmm_blocks_attend(s, r, r, r, PTR, PTR, PTR, None) == status
    assert L.spmm_blocks_backward(s, r, r, r, PTR, PTR, PTR, r, PTR, PTR, PTR, PTR, 1 << 40,
                                  None) == status
    assert L.spmm_blocks_select_workspace(s) == 0 and L.spmm_blocks_backward_workspace(s) == 0


def test_blocks_refuse_tensors(dyn):
    L, s, r = dyn.lib, shape(dyn), rows(dyn)
    big = 1 << 40
    for bad in (rows(dyn, data=0), rows(dyn, data=4104), rows(dyn, st=65), rows(dyn, sh=-64)):
        assert L.spmm_blocks_means(s, bad, -1, PTR, None) == INVALID
        assert L.spmm_blocks_select(s, bad, PTR, PTR, PTR, big, None) == INVALID
        for at in range(3):
            t = [r, r, r]
            t[at] = bad
            assert L.spmm_blocks_attend(s, *t, PTR, PTR, PTR, None) == INVALID
        assert L.spmm_blocks_backward(s, r, r, r, PTR, PTR, PTR, bad, PTR, PTR, PTR, PTR, big,
                                      None) == INVALID
    assert L.spmm_blocks_attend(s, r, r, r, None, PTR, PTR, None) == INVALID
    assert L.spmm_blocks_attend(s, r, r, r, PTR, PTR, None, None) == INVALID
    long = shape(dyn, Tk=1 << 20)                # more blocks than a row of one CTA
    assert L.spmm_blocks_select_workspace(long) > 0
    assert L.spmm_blocks_select(long, r, PTR, PTR, None, 0, None) == INVALID
    need = L.spmm_blocks_backward_workspace(s)
    assert need > 0
    assert L.spmm_blocks_backward(s, r, r, r, PTR, PTR, PTR, r, PTR, PTR, PTR, PTR, need - 1,
                                  None) == INVALID
    # widths and types of the matrix kernels
    for bad in (dict(D=32), dict(dtype=0)):
        assert L.spmm_blocks_attend(shape(dyn, **bad), r, r, r, PTR, PTR, PTR, None) == UNSUPPORTED
    # nothing to do is no error
    assert L.spmm_blocks_attend(shape(dyn, B=0), r, r, r, None, None, None, None) == 0
