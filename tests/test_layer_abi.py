"""The C ABI of the experts' products and of the heads without a GPU: argument checks on
the host, scratch sizes; and the binding's frequencies."""
import ctypes
import math

import pytest

INVALID, UNSUPPORTED = 1, 5
PTR, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4104)    # never dereferenced


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_dense_matrix_gb300.heads as heads
    return heads


def product(L, dtype=1, xs=PTR, w=PTR, se=16 * 24, sh=24, sf=1, offsets=PTR, P=8, E=3, H=16, F=24,
            ys=PTR):
    return L.spmm_routes_product(dtype, xs, w, se, sh, sf, offsets, P, E, H, F, ys, None)


def weights(L, dtype=1, xs=PTR, dys=PTR, offsets=PTR, P=8, E=3, H=16, F=24, dw=PTR, se=16 * 24,
            sh=24, sf=1, work=None, need=0):
    return L.spmm_routes_product_weights(dtype, xs, dys, offsets, P, E, H, F, dw, se, sh, sf, work,
                                         need, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), INVALID), (dict(dtype=0), UNSUPPORTED), (dict(P=-1), INVALID),
    (dict(E=-1), INVALID), (dict(H=-8), INVALID), (dict(offsets=None), INVALID),
    (dict(H=12), UNSUPPORTED), (dict(F=20), UNSUPPORTED), (dict(E=2049), UNSUPPORTED),
    (dict(P=1 << 31), UNSUPPORTED), (dict(P=(1 << 31) - 65536), UNSUPPORTED), (dict(H=1 << 21), UNSUPPORTED), (dict(F=1 << 21), UNSUPPORTED),
    (dict(xs=None), INVALID), (dict(xs=ODD), INVALID), (dict(se=-8), INVALID),
    (dict(se=4), INVALID), (dict(sh=20), INVALID), (dict(sh=24, sf=8), INVALID),
    (dict(sh=0), INVALID), (dict(sh=1, sf=0), INVALID), (dict(sh=1, sf=12), INVALID)])
def test_products_refuse(m, bad, status):
    assert product(m.lib, **bad) == status
    assert weights(m.lib, **bad) == status


def test_products_refuse_outputs(m):
    for bad in (None, ODD):
        assert product(m.lib, ys=bad) == INVALID and product(m.lib, w=bad) == INVALID
        assert weights(m.lib, dw=bad) == INVALID and weights(m.lib, dys=bad) == INVALID
    for bad in (dict(se=0), dict(sh=16), dict(sh=1, sf=8)):      # on top of one another
        assert weights(m.lib, **bad) == INVALID
    assert product(m.lib, sh=1 << 38) == UNSUPPORTED and product(m.lib, se=1 << 38) == UNSUPPORTED
    # few experts with many slots: their parts need scratch
    size = m.lib.spmm_routes_product_weights_workspace
    assert size(8, 3, 16, 24) == 0 and size(1 << 20, 64, 4096, 4096) == 0 and size(-1, 3, 16, 24) == 0
    need = size(100000, 3, 16, 24)
    assert need == 25 * 3 * 16 * 24 * 4          # 76 pairs of CTAs for three tiles
    assert weights(m.lib, P=100000) == INVALID and weights(m.lib, P=100000, work=ODD, need=need) == INVALID
    assert weights(m.lib, P=100000, work=PTR, need=need - 1) == INVALID
    # nothing to do is no error, and needs no device
    assert product(m.lib, P=0, xs=None, ys=None) == 0 and product(m.lib, F=0, ys=None) == 0
    assert weights(m.lib, E=0, dw=None) == 0 and weights(m.lib, H=0, dw=None) == 0


def shape(m, **kw):
    s = dict(B=2, T=3, Hq=4, Hk=2, D=64, R=32, dtype=1, weight_dtype=0, interleaved=0, eps=1e-6,
             magnitude=1.0, turns=4096, positions=None, p_sb=0, p_st=0, lengths=None, wq=4096,
             wk=4096)
    s.update(kw)
    return m._HeadsShape(*s.values())


def every_call(m, s, q=None, k=None, work=1 << 30, dwq=PTR, dwk=PTR, out=PTR, cache=None, v=None):
    """The statuses of the three calls."""
    L, r = m.lib, m._Rows(4096, 8192, 256, 64)
    q, k, c, v = q or r, k or r, cache or r, v or r
    t = m._HeadsShape.from_buffer_copy(s)
    if not t.positions:
        t.lengths = 4096
    return (L.spmm_heads_rotate(s, q, k, out, out, None),
            L.spmm_heads_append(t, q, k, v, out, c, c, 10, None),
            L.spmm_heads_rotate_backward(s, q, k, r, r, out, out, dwq, dwk, PTR, work, None))


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(D=0), INVALID),
    (dict(R=-16), INVALID), (dict(R=80), INVALID), (dict(dtype=3), INVALID),
    (dict(weight_dtype=2), INVALID), (dict(wq=4104), INVALID), (dict(wk=4100), INVALID),
    (dict(turns=None), INVALID), (dict(D=72), UNSUPPORTED), (dict(R=24), UNSUPPORTED),
    (dict(D=272), UNSUPPORTED), (dict(T=(1 << 26) + 1), UNSUPPORTED), (dict(Hq=65536), UNSUPPORTED),
    (dict(B=1 << 12, T=1 << 20), UNSUPPORTED), (dict(positions=4096, lengths=4096), INVALID)])
def test_heads_refuse_shapes(m, bad, status):
    s = shape(m, **bad)
    assert every_call(m, s) == (status,) * 3
    assert m.lib.spmm_heads_backward_workspace(s) == 0


def test_heads_refuse_tensors(m):
    s, R = shape(m), m._Rows
    for bad in (R(None, 0, 0, 0), R(4104, 8192, 256, 64), R(4096, 8192, 257, 64),
                R(4096, 8192, 256, -64)):
        assert every_call(m, s, q=bad) == (INVALID,) * 3
        assert every_call(m, s, k=bad) == (INVALID,) * 3
        assert every_call(m, s, cache=bad)[1] == INVALID and every_call(m, s, v=bad)[1] == INVALID
    for bad in (R(4096, 0, 256, 64), R(4096, 8192, 0, 64), R(4096, 8192, 256, 0)):
        assert every_call(m, s, cache=bad)[1] == INVALID     # rows on top of one another
    assert every_call(m, s, out=None) == (INVALID,) * 3
    assert every_call(m, s, out=ODD) == (INVALID,) * 3
    assert every_call(m, s, dwq=None)[2] == INVALID and every_call(m, s, dwk=None)[2] == INVALID
    need = m.lib.spmm_heads_backward_workspace(s)
    assert need > 0 and every_call(m, s, work=need - 1)[2] == INVALID
    assert m.lib.spmm_heads_backward_workspace(shape(m, wq=None, wk=None)) == 0
    r = R(4096, 8192, 256, 64)
    assert m.lib.spmm_heads_append(s, r, r, r, PTR, r, r, 10, None) == INVALID   # no lengths
    t = shape(m, lengths=4096)
    assert m.lib.spmm_heads_append(t, r, r, r, PTR, r, r, -1, None) == INVALID
    assert m.lib.spmm_heads_append(t, r, r, r, PTR, r, r, 1 << 27, None) == UNSUPPORTED
    # nothing to do is no error
    none = R(None, 0, 0, 0)
    assert m.lib.spmm_heads_rotate(shape(m, B=0), none, none, None, None, None) == 0


def test_frequencies(m):
    """Each scaling's fastest and slowest pairs, and what lies between."""
    R, base = 64, 1e4
    plain, one = m._frequencies(R, base, None)
    assert one == 1.0 and plain[0] == 1.0
    assert all(abs(f * base ** (2 * i / R) - 1) < 1e-14 for i, f in enumerate(plain))
    linear, _ = m._frequencies(R, base, {"kind": "linear", "factor": 4.0})
    assert all(f == p / 4 for f, p in zip(linear, plain))
    slow, _ = m._frequencies(R, base, {"kind": "base", "factor": 4.0})
    assert slow[0] == 1.0 and abs(slow[-1] * 4 / plain[-1] - 1) < 1e-14
    L = 4096
    for how in ({"kind": "parts"}, {"kind": "bands"}):
        f, size = m._frequencies(R, base, {**how, "factor": 8.0, "original_length": L})
        assert size == (1.0 if how["kind"] == "bands" else 0.1 * math.log(8) + 1)
        ratio = [p / x for p, x in zip(plain, f)]
        assert ratio[0] == 1 and abs(ratio[-1] - 8) < 1e-12
        assert all(a <= b + 1e-12 for a, b in zip(ratio, ratio[1:]))
        assert any(1.1 < x < 7.9 for x in ratio)
        for p, x in zip(plain, ratio):
            turns = L * p / math.tau
            if turns > 45:
                assert x == 1
            if turns < 0.7:
                assert abs(x - 8) < 1e-12


@pytest.mark.parametrize("bad", [
    {"kind": "cubic", "factor": 2.0}, {"factor": 2.0}, {"kind": "linear"},
    {"kind": "linear", "factor": 0.0}, {"kind": "linear", "factor": float("inf")},
    {"kind": "parts", "factor": 2.0}, {"kind": "bands", "factor": 2.0, "original_length": 0},
    {"kind": "linear", "factor": 2.0, "slow": 1.0},
    {"kind": "bands", "factor": 2.0, "original_length": 100, "fast": 1.0, "slow": 1.0}])
def test_scalings_refused(m, bad):
    with pytest.raises(ValueError):
        m._frequencies(64, 1e4, bad)


@pytest.mark.parametrize("kw", [
    dict(dim=72), dict(dim=272), dict(dim=0), dict(dim=64, rotary_dim=24),
    dict(dim=64, rotary_dim=80), dict(dim=64, rotary_dim=-16), dict(dim=64, layout="thirds"),
    dict(dim=64, base=1.0), dict(dim=64, base=float("nan")), dict(dim=64, frequencies=[1.0]),
    dict(dim=32, frequencies=[float("inf")] * 16), dict(dim=64, device="cpu"),
    dict(dim=32, frequencies=[1.0] * 16, scaling={"kind": "linear", "factor": 2.0})])
def test_rotations_refused(m, kw):
    with pytest.raises(ValueError):
        m.HeadRotation(**kw)


def test_public_names(m):
    import sparse_dense_matrix_gb300 as sdm
    assert "HeadRotation" in sdm.__all__ and sdm.HeadRotation is m.HeadRotation
