"""Expert routes on the GPU against a plain 64-bit form: the sort exactly, the
gathered rows bit for bit, weighted sums and gradients within the bound of fp32
sums rounded once."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import dynamic_ref as ref  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


def make_ids(T, k, E, seed, drop=0.0, skew=False):
    g = torch.Generator().manual_seed(seed)
    if E == 0:
        return torch.full((T, k), -1, dtype=torch.int32)
    ids = torch.randint(E, (T, k), generator=g)
    if skew:
        ids = torch.where(torch.rand(T, k, generator=g) < 0.9, min(3, E - 1), ids)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    return ids.to(torch.int32)


@pytest.mark.parametrize("T,k,E,drop,skew", [
    (1, 1, 1, 0, False), (1, 8, 64, 0, False), (7, 3, 5, 0.3, False), (33, 2, 2048, 0, False),
    (1024, 8, 128, 0, False),      # the last size of the single launch
    (1025, 8, 128, 0.1, False),    # the first of two launches
    (4097, 5, 300, 0, True), (20000, 2, 17, 0.02, True), (100, 4, 8, 1.0, False),
    (50, 2, 0, 0, False)])
def test_sort(sdm, cuda_device, T, k, E, drop, skew):
    ids = make_ids(T, k, E, T + E, drop, skew)
    offsets, slots = ref.routes(ids, E)
    r = sdm.ExpertRoutes(ids.to(cuda_device), E)
    assert torch.equal(r.offsets.cpu(), offsets)
    assert torch.equal(r.slots.cpu(), slots)


def test_sort_drops_ids_out_of_range(sdm, cuda_device):
    ids = torch.tensor([[5, -7], [2, 4], [2 ** 31 - 1, 0]], dtype=torch.int32)
    r = sdm.ExpertRoutes(ids.to(cuda_device), 4)
    assert r.slots.cpu().tolist() == [[-1, -1], [1, -1], [-1, 0]]
    assert r.offsets.cpu().tolist() == [0, 1, 1, 2, 2]


SHAPES = [(1, 1, 1, 1), (3, 2, 4, 8), (5, 8, 16, 64), (37, 3, 7, 1001), (64, 4, 9, 2048),
          (130, 2, 8, 520), (9, 6, 300, 4104), (2, 1, 3, 12345), (300, 9, 11, 36)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.25, 1.0])
def test_products_and_gradients(sdm, cuda_device, T, k, E, H, dtype, drop):
    dt = DT[dtype]
    ids = make_ids(T, k, E, H, drop)
    _, slots = ref.routes(ids, E)
    slots = slots.to(cuda_device)
    g = torch.Generator(device=cuda_device).manual_seed(H)
    rnd = lambda *s: torch.randn(*s, generator=g, device=cuda_device).to(dt)  # noqa: E731
    x, y, dout, dxs = rnd(T, H), rnd(T * k, H), rnd(T, H), rnd(T * k, H)
    w = torch.rand(T, k, generator=g, device=cuda_device)
    r = sdm.ExpertRoutes(ids.to(cuda_device), E)
    R, P = ref.matrix(slots, w), ref.matrix(slots, torch.ones_like(w))
    u, tiny = ref.U[dt], ref.TINY[dt]

    assert torch.equal(r.dispatch(x).double(), P.T @ x.double())   # a copy: exact

    want = R @ y.double()
    tol = u * want.abs() + 2 * (k + 1) * ref.E32 * (R @ y.double().abs()) + tiny
    ref.close(r.combine(y, w), want, tol, "combine")

    want = P @ dxs.double()
    tol = u * want.abs() + 2 * (k + 1) * ref.E32 * (P @ dxs.double().abs()) + tiny
    ref.close(r.dispatch_backward(dxs), want, tol, "dispatch_backward")

    dy, dw = r.combine_backward(dout, y, w)
    want = R.T @ dout.double()
    ref.close(dy, want, (u + 2 * ref.E32) * want.abs() + tiny, "dy")
    at = slots.clamp(min=0).long()
    pairs = dout.double()[:, None] * y.double()[at]
    kept = (slots >= 0)[..., None]
    want = torch.where(kept, pairs, 0.0).sum(-1)
    ref.close(dw, want, 2 * H * ref.E32 * torch.where(kept, pairs, 0.0).abs().sum(-1), "dweights")
    dy1, none = r.combine_backward(dout, y)
    assert none is None and torch.equal(dy1.double(), P.T @ dout.double())


def test_gradients_against_differences(sdm, cuda_device):
    """combine is linear in y and in w, so central differences of its 64-bit form
    are exact but for their own rounding (about 1e-9 here): the gradients must
    match them to within their fp32 bounds."""
    T, k, E, H = 11, 3, 5, 24
    ids = make_ids(T, k, E, 1, 0.2)
    r = sdm.ExpertRoutes(ids.to(cuda_device), E)
    g = torch.Generator(device=cuda_device).manual_seed(5)
    y, dout = (torch.randn(n, H, generator=g, device=cuda_device) for n in (T * k, T))
    w = torch.rand(T, k, generator=g, device=cuda_device)

    def loss(y_, w_):
        return (ref.matrix(r.slots, w_) @ y_ * dout.double()).sum()

    dy, dw = r.combine_backward(dout, y, w)
    step = 2.0 ** -10
    for i in range(20):
        ty = torch.randn(y.shape, generator=g, device=cuda_device).double()
        tw = torch.randn(w.shape, generator=g, device=cuda_device).double()
        up = loss(y.double() + step * ty, w.double()) - loss(y.double() - step * ty, w.double())
        used = torch.zeros(T * k, 1, dtype=torch.float64, device=cuda_device)
        used[r.slots[r.slots >= 0].long()] = 1
        tol = 4 * ref.E32 * (dy.double() * ty).abs().sum() + 1e-9
        assert abs(up / (2 * step) - (dy.double() * ty * used).sum()) <= tol
        up = loss(y.double(), w.double() + step * tw) - loss(y.double(), w.double() - step * tw)
        mag = (dout.double().abs() @ y.double().abs().T).max() * tw.abs().sum()
        assert abs(up / (2 * step) - (dw.double() * tw).sum()) <= 2 * H * ref.E32 * mag + 1e-9


def test_dropped_rows_are_never_read(sdm, cuda_device):
    """NaN in the rows past the kept pairs, and an infinite weight on a dropped pair."""
    ids = torch.tensor([[0, -1], [-1, -1], [1, 0]], dtype=torch.int32, device=cuda_device)
    r = sdm.ExpertRoutes(ids, 2)
    y = torch.ones(6, 16, device=cuda_device, dtype=torch.bfloat16)
    y[3:] = float("nan")
    w = torch.tensor([[2.0, float("inf")], [float("nan"), 1.0], [1.0, 0.5]], device=cuda_device)
    assert r.combine(y, w)[:, 0].tolist() == [2.0, 0.0, 1.5]
    dy, dw = r.combine_backward(torch.ones(3, 16, device=cuda_device, dtype=torch.bfloat16), y, w)
    assert dy[:, 0].tolist() == [2.0, 0.5, 1.0, 0.0, 0.0, 0.0]
    assert dw.tolist() == [[16.0, 0.0], [0.0, 0.0], [16.0, 16.0]]


@pytest.mark.parametrize("dtype", list(DT))
def test_strided_and_unaligned_rows(sdm, cuda_device, dtype):
    dt = DT[dtype]
    T, k, E, H = 21, 2, 4, 64
    ids = make_ids(T, k, E, 3).to(cuda_device)
    r = sdm.ExpertRoutes(ids, E)
    big = torch.randn(T, 3 * H + 1, device=cuda_device).to(dt)
    y = torch.randn(T * k, H, device=cuda_device).to(dt)
    w = torch.rand(T, k, device=cuda_device)
    for x in (big[:, :H], big[:, 1:H + 1], big[:, H:2 * H], big[:1, :H].expand(T, H)):
        assert torch.equal(r.dispatch(x), r.dispatch(x.contiguous()))
        a, b = r.combine_backward(x, y, w), r.combine_backward(x.contiguous(), y, w)
        assert torch.equal(a[0], b[0])
        ref.close(a[1], b[1], 4 * H * ref.E32 * (x.abs().max() * y.abs().max() * H).double(), "dw")


def test_empty(sdm, cuda_device):
    for T, k, H in ((0, 2, 8), (3, 0, 8), (3, 2, 0)):
        r = sdm.ExpertRoutes(torch.zeros(T, k, dtype=torch.int32, device=cuda_device), 2)
        x = torch.ones(T, H, device=cuda_device)
        xs = r.dispatch(x)
        assert xs.shape == (T * k, H)
        out = r.combine(xs, torch.ones(T, k, device=cuda_device))
        assert out.shape == (T, H) and (out == (k if k else 0)).all()
        dy, dw = r.combine_backward(x, xs, torch.ones(T, k, device=cuda_device))
        assert dy.shape == (T * k, H) and dw.shape == (T, k) and (dw == H).all()


def test_rows_past_32_bit_offsets(sdm, cuda_device):
    """2.3e9 elements by slot: the last rows are where 32-bit offsets would wrap."""
    T, k, H = 70000, 8, 4104
    ids = torch.zeros(T, k, dtype=torch.int32, device=cuda_device)
    r = sdm.ExpertRoutes(ids, 1)
    x = (torch.arange(T, device=cuda_device) % 251).to(torch.bfloat16)[:, None].expand(T, H)
    x = x.contiguous()
    xs = r.dispatch(x)
    assert torch.equal(xs[-8:], x[-1:].expand(8, H)) and torch.equal(xs[8 * 65432], x[65432])
    out = r.combine(xs)
    assert torch.equal(out[-3:], (8 * x[-3:].float()).to(torch.bfloat16))


def test_reproducible_and_streams(sdm, cuda_device):
    T, k, E, H = 3000, 4, 32, 1024
    side = torch.cuda.Stream()
    main = None
    for stream in (None, side):
        with torch.cuda.stream(side if stream is not None else torch.cuda.current_stream()):
            g = torch.Generator(device=cuda_device).manual_seed(9)
            ids = torch.randint(E, (T, k), generator=g, device=cuda_device).to(torch.int32)
            x = torch.randn(T, H, generator=g, device=cuda_device).to(torch.float16)
            w = torch.rand(T, k, generator=g, device=cuda_device)
        r = sdm.ExpertRoutes(ids, E, stream=stream)
        xs = r.dispatch(x, stream=stream)
        got = (r.slots, r.offsets, xs, r.combine(xs, w, stream=stream),
               *r.combine_backward(x, xs, w, stream=stream), r.dispatch_backward(xs, stream=stream))
        torch.cuda.synchronize()
        if main is None:
            main = got
        assert all(torch.equal(a, b) for a, b in zip(main, got))


def test_graph_capture(sdm, cuda_device):
    T, k, E, H = 64, 2, 8, 256
    ids = torch.randint(E, (T, k), device=cuda_device).to(torch.int32)
    x = torch.randn(T, H, device=cuda_device, dtype=torch.bfloat16)
    w = torch.rand(T, k, device=cuda_device)

    def step():
        r = sdm.ExpertRoutes(ids, E)
        return r.combine(r.dispatch(x), w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    ids.copy_(torch.randint(E, (T, k), device=cuda_device))
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, step())


def test_refusals(sdm, cuda_device):
    ids = torch.zeros(4, 2, dtype=torch.int32, device=cuda_device)
    with pytest.raises(TypeError):
        sdm.ExpertRoutes(ids.long(), 4)
    with pytest.raises(ValueError):
        sdm.ExpertRoutes(ids.cpu(), 4)
    with pytest.raises(ValueError):
        sdm.ExpertRoutes(ids[0], 4)
    with pytest.raises(ValueError):
        sdm.ExpertRoutes(ids[:, :1], 4)
    with pytest.raises(ValueError):
        sdm.ExpertRoutes(ids, 2049)
    r = sdm.ExpertRoutes(ids, 4)
    x, y = torch.ones(4, 8, device=cuda_device), torch.ones(8, 8, device=cuda_device)
    w = torch.ones(4, 2, device=cuda_device)
    with pytest.raises(ValueError):
        r.dispatch(x[:3])
    with pytest.raises(TypeError):
        r.dispatch(x.double())
    with pytest.raises(ValueError):
        r.dispatch(x.t().contiguous().t()[:, ::2])
    with pytest.raises(ValueError):
        r.combine(y[:7], w)
    with pytest.raises(TypeError):
        r.combine(y, w.half())
    with pytest.raises(ValueError):
        r.combine(y, w[:, :1])
    with pytest.raises(TypeError):
        r.combine_backward(x.half(), y, w)
    with pytest.raises(ValueError):
        r.combine_backward(x, y[:, :4], w)
    # the context is intact
    assert (r.combine(y, w) == 2).all()
