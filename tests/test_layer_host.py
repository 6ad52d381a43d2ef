"""The binding of the experts' products and of the heads without a GPU: the library's calls are
stood in for, and tensors are the host's."""
import copy
import math
import pickle
import weakref

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dynamic():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_dense_matrix_gb300.dynamic as dynamic
    return dynamic


class Calls:
    """The library, with some of its calls replaced."""

    def __init__(self, lib, **calls):
        self._lib = lib
        self.__dict__.update(calls)

    def __getattr__(self, name):
        return getattr(self._lib, name)


def host_routes(dynamic, monkeypatch, T, k, E):
    """Routes whose tensors are the host's, and a binding that takes such."""
    monkeypatch.setattr(dynamic, "_elsewhere", lambda dev, stream: None)
    monkeypatch.setattr(dynamic, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(dynamic, "_tensor", lambda t, *a, **kw: t)
    r = dynamic.ExpertRoutes.__new__(dynamic.ExpertRoutes)
    r.device, r.num_experts, r.T, r.k, r._stream = torch.device("cpu"), E, T, k, 0
    r.slots = torch.zeros(T, k, dtype=torch.int32)
    r.offsets = torch.zeros(E + 1, dtype=torch.int32)
    r._routes = (r.slots.data_ptr(), r.offsets.data_ptr(), T, k, E)
    return r


def test_gradients_scratch_is_held_until_its_last_launch(dynamic, monkeypatch):
    """A tensor that nothing refers to goes back to the allocator: another thread on the same
    stream could be given the scratch of the matrices' gradient before it is used."""
    T, E, H, F = 5000, 1, 72, 264
    need = dynamic.lib.spmm_routes_product_weights_workspace(T, E, H, F)
    assert need > 0
    routes = host_routes(dynamic, monkeypatch, T, 1, E)
    made, seen, empty = [], [], torch.empty

    def make(*args, **kw):
        t = empty(*args, **kw)
        if t.dtype == torch.uint8:
            made.append((weakref.ref(t), t.data_ptr()))
        return t

    def launch(name):
        def call(*args):
            assert len(made) == 1 and made[0][0]() is not None, f"{name}: the scratch is gone"
            seen.append(name)
            if name == "weights":
                assert args[-3:-1] == (made[0][1], need)
            return 0
        return call

    monkeypatch.setattr(dynamic, "lib", Calls(dynamic.lib, spmm_routes_product=launch("rows"),
                                              spmm_routes_product_weights=launch("weights")))
    monkeypatch.setattr(torch, "empty", make)
    xs, grad = (torch.zeros(T, n, dtype=torch.bfloat16) for n in (H, F))
    routes.product_backward(grad, xs, torch.zeros(E, H, F, dtype=torch.bfloat16))
    assert seen == ["rows", "weights"]


@pytest.mark.parametrize("E,H,F", [(1, 8, 8), (152, 8, 8), (160, 256, 256), (2048, 64, 64),
                                   (8, 1024, 1024), (3, 4096, 8)])
def test_no_part_of_the_gradient_is_longer_than_its_waits(dynamic, E, H, F):
    """One expert may hold all of the slots. 64 of them take 0.31 us, a wait gives up after
    0.5 s: parts of at most 2^24 slots keep to a sixth of that."""
    size = dynamic.lib.spmm_routes_product_weights_workspace
    for P in (1 << 24, (1 << 24) + 1, 1 << 28, (1 << 31) - 65537):
        parts = max(1, size(P, E, H, F) // (E * H * F * 4))
        assert -(-P // parts) <= 1 << 24, (P, parts)


def copies(x):
    """x copied, copied whole, and written out and read again."""
    return copy.copy(x), copy.deepcopy(x), pickle.loads(pickle.dumps(x))


def first_use_lends(module, monkeypatch, x, tensors):
    """A copy's tensors may be the original's, of another stream's memory: the first stream that
    uses them is lent them, whichever it is, and others each time."""
    lent = []
    monkeypatch.setattr(module, "_lent", lambda dev, *t: lent.append(t))
    for stream, count in ((0, 1), (0, 1), (7, 2), (7, 3), (0, 3)):
        monkeypatch.setattr(module, "_raw_stream", lambda index: stream)
        assert x._on_stream() == stream and len(lent) == count
        assert len(lent[-1]) == len(tensors) and all(a is b for a, b in zip(lent[-1], tensors))


def test_copies_of_routes_use_their_own_tensors(dynamic, monkeypatch):
    """Not the original's, which may be gone by the time the copy is used."""
    routes = host_routes(dynamic, monkeypatch, 7, 2, 3)
    for r in copies(routes):
        assert r._routes == (r.slots.data_ptr(), r.offsets.data_ptr(), 7, 2, 3)
        assert torch.equal(r.slots, routes.slots) and r.device == routes.device
        first_use_lends(dynamic, monkeypatch, r, [r.slots, r.offsets])


@pytest.mark.parametrize("rotary", [64, 0])
def test_copies_of_a_rotation_use_their_own_frequencies(dynamic, monkeypatch, rotary):
    import sparse_dense_matrix_gb300.heads as heads
    monkeypatch.setattr(heads, "_raw_stream", lambda index: 0)
    rot = heads.HeadRotation.__new__(heads.HeadRotation)
    rot.turns, rot.dim, rot.rotary_dim = torch.arange(rotary // 2), 64, rotary
    rot.device, rot._turns, rot._stream = rot.turns.device, rot.turns.data_ptr() or None, 0
    for r in copies(rot):
        assert r._turns == (r.turns.data_ptr() or None) and torch.equal(r.turns, rot.turns)
        assert r.dim == 64
        first_use_lends(heads, monkeypatch, r, [r.turns])


@pytest.mark.parametrize("lengths", ["none", "behind the lists", "asked for", "given"])
def test_copies_of_a_selection_use_their_own_lists(dynamic, monkeypatch, lengths):
    monkeypatch.setattr(dynamic, "_raw_stream", lambda index: 0)
    B, Tq, Hk, n = shape = (3, 2, 2, 4)
    size = B * Tq * Hk * n
    sel = dynamic.BlockSelection.__new__(dynamic.BlockSelection)
    own = lengths in ("behind the lists", "asked for")
    mem = torch.arange(size + 3, dtype=torch.int32) if own else \
        torch.arange(size, dtype=torch.int32).view(shape)
    sel._set(mem, shape, 16, 100, True)
    if own:
        sel._lengths = sel._lists + 4 * size
        if lengths == "asked for":
            assert sel.lengths.tolist() == [size, size + 1, size + 2]
    elif lengths == "given":
        sel._keep(torch.tensor([5, 6, 7], dtype=torch.int32))
    for s in copies(sel):
        assert s._lists == s._mem.data_ptr() and torch.equal(s.blocks, sel.blocks)
        if lengths == "none":
            assert s._lengths is None and s.lengths is None
        else:
            assert s._lengths == s.lengths.data_ptr() and torch.equal(s.lengths, sel.lengths)
        assert s.num_keys == 100
        first_use_lends(dynamic, monkeypatch, s, [s._mem, s._kept])


@pytest.mark.parametrize("how", [
    {"kind": "parts", "slow": 0.0}, {"kind": "parts", "slow": -1.0}, {"kind": "parts", "fast": 0.0},
    {"kind": "parts", "fast": 0.5}, {"kind": "parts", "fast": math.inf},
    {"kind": "parts", "fast": math.nan}, {"kind": "parts", "slow": math.nan},
    {"kind": "parts", "original_length": math.inf}, {"kind": "bands", "original_length": math.inf},
    {"kind": "parts", "magnitude": math.nan}])
def test_scalings_without_a_meaning_are_refused(dynamic, how):
    import sparse_dense_matrix_gb300 as sdm
    with pytest.raises(ValueError, match="scaling|magnitude"):
        sdm.HeadRotation(64, scaling={"factor": 2.0, "original_length": 4096, **how})


@pytest.mark.parametrize("magnitude", [math.nan, math.inf])
def test_magnitude_is_finite(dynamic, magnitude):
    import sparse_dense_matrix_gb300 as sdm
    with pytest.raises(ValueError, match="magnitude"):
        sdm.HeadRotation(64, magnitude=magnitude)


def test_parts_between_equal_numbers_of_turns(dynamic):
    """A step between two neighbouring pairs."""
    import sparse_dense_matrix_gb300.heads as heads
    how = {"kind": "parts", "factor": 8.0, "original_length": 4096, "fast": 8.0, "slow": 8.0}
    f, _ = heads._frequencies(64, 1e4, how)
    plain, _ = heads._frequencies(64, 1e4, None)
    turns = [4096 * p / math.tau for p in plain]
    assert all(x == p for x, p, t in zip(f, plain, turns) if t > 8.0)
    assert all(abs(x * 8 / p - 1) < 1e-14 for x, p, t in zip(f, plain, turns) if t < 8.0)


def test_caches_in_one_place_are_refused(dynamic, monkeypatch):
    """Keys and values would be written over one another."""
    import ctypes
    import sparse_dense_matrix_gb300.heads as heads
    R, out = heads._Rows, ctypes.c_void_p(4096)              # (never read)
    s = heads._HeadsShape(2, 3, 4, 2, 64, 32, 1, 0, 0, 1e-6, 1.0, 4096, None, 0, 0, 4096, None, None)
    r, c, d = (R(4096 << i, 8192, 256, 64) for i in (0, 10, 20))
    append = heads.lib.spmm_heads_append
    assert append(s, r, r, r, out, c, c, 10, None) == 1
    for bad in (R(None, 0, 0, 0), R(4104, 8192, 256, 64), R(4096, 0, 256, 64), R(4096, 8192, 0, 64),
                R(4096, 8192, 256, 0)):                      # the others' checks stand
        assert append(s, r, r, r, out, bad, d, 10, None) == 1
        assert append(s, r, r, r, out, c, bad, 10, None) == 1

    # the binding's own message, before the library is called
    monkeypatch.setattr(heads, "_elsewhere", lambda dev, stream: None)
    monkeypatch.setattr(heads, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(dynamic, "_tensor", lambda t, *a, **kw: t)
    calls = []
    monkeypatch.setattr(heads, "lib", Calls(heads.lib, spmm_heads_append=lambda *a: calls.append(a)))
    rot = heads.HeadRotation.__new__(heads.HeadRotation)
    rot.turns, rot.dim, rot.rotary_dim, rot.magnitude = torch.zeros(32).long(), 64, 64, 1.0
    rot._interleaved, rot._weight_shape = 0, (64,)
    rot._tell(0)
    q, k, v = (torch.zeros(2, 1, n, 64) for n in (4, 2, 2))
    ck, L = torch.zeros(2, 8, 2, 64), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="in one place"):
        rot.append(q, k, v, ck, ck, L)
    assert not calls
    both = torch.zeros(2, 8, 2, 2, 64)                       # side by side is another thing
    rot.append(q, k, v, both[:, :, 0], both[:, :, 1], L)
    rot.append(q, k, v, ck[:, :0], ck[:, :0], L)             # and no rows have no place
    assert len(calls) == 2


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, pickle.dumps])
def test_plans_are_not_copied(dynamic, how):
    """Two of them would free one plan."""
    import sparse_dense_matrix_gb300 as sdm
    adj = sdm.SparseAdj.__new__(sdm.SparseAdj)
    adj._plan = adj._t = adj._tmean = None
    with pytest.raises(TypeError, match="cannot be copied"):
        how(adj)
