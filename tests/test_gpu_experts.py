"""The experts' products on the GPU against plain 64-bit products.

The products of two 16-bit values are exact in fp32; a sum of n of them in fp32, in any
order, is off by at most (n + 32) 2^-24 times the sum of magnitudes (32: what a matrix
instruction may cut off where it aligns the terms of one step), and is rounded once."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import dynamic_ref as ref  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


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


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


def matrices(dev, seed, E, H, F, dt, stored):
    w = (randn(dev, seed, E, H, F) * H ** -0.5).to(dt)
    if stored == "out_in":
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    return w


def tolerance(want, mag, n, dt):
    return ref.U[dt] * want.abs() + (n + 32) * ref.E32 * mag + ref.TINY[dt]


def expected(offsets, xs, w, dys=None):
    """ys (and dxs, dw) in 64 bits, each with its tolerance."""
    at, dt = offsets.tolist(), xs.dtype
    (P, H), F = xs.shape, w.shape[2]
    kw = {"dtype": torch.float64, "device": xs.device}
    r = [torch.zeros(P, F, **kw)] + ([torch.zeros(P, H, **kw), torch.zeros(w.shape, **kw)]
                                     if dys is not None else [])
    tol = [torch.zeros_like(x) for x in r]

    def put(i, rows, a, b, n):
        r[i][rows] = a @ b
        tol[i][rows] = tolerance(r[i][rows], a.abs() @ b.abs(), n, dt)

    for e in range(w.shape[0]):
        rows = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        x, we = xs[rows].double(), w[e].double()
        put(0, rows, x, we, H)
        if dys is not None:
            dy = dys[rows].double()
            put(1, rows, dy, we.T, F)
            put(2, e, x.T, dy, at[e + 1] - at[e])
    return list(zip(r, tol))


SHAPES = [
    (1, 1, 1, 8, 8, 0.0, False), (1, 8, 64, 64, 72, 0.0, False), (3, 2, 4, 136, 40, 0.3, False),
    (37, 3, 7, 1000, 520, 0.05, False), (64, 4, 9, 256, 128, 0.0, False),
    (300, 2, 3, 512, 264, 0.0, False), (130, 2, 8, 72, 1032, 0.1, False),
    (700, 3, 5, 320, 256, 0.0, True), (40, 2, 300, 64, 64, 0.0, False),
    (100, 4, 8, 192, 48, 1.0, False), (2048, 2, 2, 128, 128, 0.02, False),
    (17, 1, 2048, 16, 24, 0.0, False), (1500, 1, 1, 2056, 136, 0.0, False),
    (515, 2, 4, 640, 384, 0.0, False)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("stored", ["in_out", "out_in"])
@pytest.mark.parametrize("T,k,E,H,F,drop,skew", SHAPES)
def test_products_and_gradients(sdm, cuda_device, T, k, E, H, F, drop, skew, stored, dtype):
    dt = DT[dtype]
    routes = sdm.ExpertRoutes(make_ids(T, k, E, T + H, drop, skew).to(cuda_device), E)
    xs, dys = (randn(cuda_device, 1 + i, T * k, n).to(dt) for i, n in enumerate((H, F)))
    kept = int(routes.offsets[-1])
    xs[kept:] = dys[kept:] = float("nan")        # rows of no pair may hold anything
    w = matrices(cuda_device, 3, E, H, F, dt, stored)
    got = [routes.product(xs, w), *routes.product_backward(dys, xs, w)]
    assert got[2].stride() == w.stride()
    for name, g, (want, tol) in zip(("ys", "dxs", "dw"), got,
                                    expected(routes.offsets, xs, w, dys)):
        assert g.dtype == dt
        ref.close(g, want, tol, name)
    assert not got[0][kept:].any() and not got[1][kept:].any()
    sdm.dynamic_sync()


@pytest.mark.parametrize("stored", ["in_out", "out_in"])
def test_one_experts_values_stay_with_it(sdm, cuda_device, stored):
    """NaN and infinities in an expert's rows or matrix do not reach the others'."""
    T, k, E, H, F, dt = 333, 1, 6, 200, 328, torch.bfloat16
    ids = make_ids(T, k, E, 5)
    routes = sdm.ExpertRoutes(ids.to(cuda_device), E)
    at = routes.offsets.tolist()
    xs, dys = (randn(cuda_device, 1 + i, T, n).to(dt) for i, n in enumerate((H, F)))
    w = matrices(cuda_device, 3, E, H, F, dt, stored)
    clean = [routes.product(xs, w), *routes.product_backward(dys, xs, w)]
    bad = 2
    xs[at[bad]:at[bad + 1]] = float("nan")
    dys[at[bad]:at[bad + 1]] = float("inf")
    w[bad] = float("nan")
    got = [routes.product(xs, w), *routes.product_backward(dys, xs, w)]
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        for i, part in ((0, rows), (1, rows), (2, e)):
            if e == bad:
                assert torch.isnan(got[i][part]).all()
            else:
                assert torch.equal(got[i][part], clean[i][part])
    # one infinity is in its own row's sums only, and one row's gradient
    xs = randn(cuda_device, 9, T, H).to(dt)
    w = matrices(cuda_device, 3, E, H, F, dt, stored)
    xs[at[1], 3] = float("inf")
    ys = routes.product(xs, w)
    assert not torch.isfinite(ys[at[1]]).any()
    ys[at[1]] = 0
    assert torch.isfinite(ys).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_strided_and_shared_matrices(sdm, cuda_device, dtype):
    dt, T, k, E, H, F = DT[dtype], 90, 2, 5, 136, 72
    routes = sdm.ExpertRoutes(make_ids(T, k, E, 1, 0.1).to(cuda_device), E)
    xs, dys = (randn(cuda_device, 1 + i, T * k, n).to(dt) for i, n in enumerate((H, F)))
    big = randn(cuda_device, 4, E, H + 8, 2 * F).to(dt)
    forms = {"columns": big[:, :H, F:],
             "columns, transposed": randn(cuda_device, 6, E, F, H + 24).to(dt)[..., :H].transpose(1, 2),
             "one for all": big[:1, :H, :F].expand(E, H, F),
             "experts in the middle": randn(cuda_device, 5, H, E, F).to(dt).transpose(0, 1)}
    for name, w in forms.items():
        got = [routes.product(xs, w), *routes.product_backward(dys, xs, w)]
        for g, (want, tol) in zip(got, expected(routes.offsets, xs, w, dys)):
            ref.close(g, want, tol, name)


def test_gradients_against_differences(sdm, cuda_device):
    """Small whole numbers: every sum is exact, and so is a difference of two results."""
    T, k, E, H, F, dt = 20, 2, 3, 16, 24, torch.float16
    g = torch.Generator().manual_seed(3)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g).to(cuda_device, dt)

    routes = sdm.ExpertRoutes(make_ids(T, k, E, 1, 0.2).to(cuda_device), E)
    xs, w, grad = whole(T * k, H), whole(E, H, F), whole(T * k, F)

    def loss(xs, w):
        return (routes.product(xs, w).double() * grad.double()).sum().item()

    dxs, dw = routes.product_backward(grad, xs, w)
    base = loss(xs, w)
    for t, d in ((xs, dxs), (w, dw)):
        for i in torch.randint(t.numel(), (60,), generator=g).tolist():
            t.view(-1)[i] += 1
            assert loss(xs, w) - base == d.view(-1)[i].item()
            t.view(-1)[i] -= 1


def test_with_the_routes(sdm, cuda_device):
    """dispatch, two products and combine, with every gradient, as one function of x."""
    T, k, E, H, F, dt = 75, 3, 6, 64, 120, torch.bfloat16
    ids = make_ids(T, k, E, 4, 0.1).to(cuda_device)
    x, dout = (randn(cuda_device, i, T, H).to(dt) for i in (1, 2))
    weights = torch.softmax(randn(cuda_device, 3, T, k), 1)
    w1, w2 = matrices(cuda_device, 4, E, H, F, dt, "in_out"), matrices(cuda_device, 5, E, F, H, dt,
                                                                       "out_in")

    def step():
        routes = sdm.ExpertRoutes(ids, E)
        xs = routes.dispatch(x)
        h = routes.product(xs, w1)
        a = torch.relu(h)
        ys = routes.product(a, w2)
        out = routes.combine(ys, weights)
        dys, dweights = routes.combine_backward(dout, ys, weights)
        da, dw2 = routes.product_backward(dys, a, w2)
        dxs, dw1 = routes.product_backward(torch.where(h > 0, da, 0), xs, w1)
        return out, routes.dispatch_backward(dxs), dw1, dw2, dweights

    got = step()
    leaves = [t.double().requires_grad_() for t in (x, w1, w2, weights)]
    xd, w1d, w2d, wd = leaves
    out = torch.zeros(T, H, dtype=torch.float64, device=cuda_device)
    for j in range(k):
        at = (ids[:, j] >= 0).nonzero()[:, 0]
        e = ids[at, j].long()
        y = torch.einsum("tf,tfh->th", torch.relu(torch.einsum("th,thf->tf", xd[at], w1d[e])), w2d[e])
        out = out.index_add(0, at, wd[at, j, None] * y)
    dx, dw1, dw2, dwt = torch.autograd.grad(out, leaves, dout.double())
    # each of up to five steps is rounded to bf16: 8 roundings of the largest values cover it
    for g, want in zip(got, (out, dx, dw1, dw2, dwt)):
        ref.close(g, want, 8 * ref.U[dt] * want.abs().max().item())
    # and the same as a captured graph, whose inputs change
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    ids.copy_(make_ids(T, k, E, 40, 0.3))
    x.copy_(randn(cuda_device, 50, T, H))
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    assert all(torch.equal(a, b) for a, b in zip(kept, again))
    sdm.dynamic_sync()


def test_rows_past_32_bit_offsets(sdm, cuda_device):
    """Elements past 2^31 of xs, of ys and of the rows' gradients."""
    T, E, H, F, dt = 300000, 2, 8192, 16, torch.bfloat16
    ids = (torch.arange(T, dtype=torch.int32)[:, None] >= 250000).to(torch.int32)
    routes = sdm.ExpertRoutes(ids.to(cuda_device), E)
    xs = torch.zeros(T, H, dtype=dt, device=cuda_device)
    w = randn(cuda_device, 1, E, H, F).to(dt)
    some = torch.tensor([0, 131072, 249999, 250000, 262144, 299999], device=cuda_device)
    xs[some] = randn(cuda_device, 2, len(some), H).to(dt)
    ys = routes.product(xs, w)
    want = torch.stack([xs[s].double() @ w[int(s >= 250000)].double() for s in some])
    mag = torch.stack([xs[s].double().abs() @ w[int(s >= 250000)].double().abs() for s in some])
    ref.close(ys[some], want, tolerance(want, mag, H, dt))
    ys[some] = 0
    assert not ys.any()
    grad = torch.zeros(T, F, dtype=dt, device=cuda_device)
    grad[some] = randn(cuda_device, 3, len(some), F).to(dt)
    dxs, dw = routes.product_backward(grad, xs, w)
    want = torch.stack([w[int(s >= 250000)].double() @ grad[s].double() for s in some])
    mag = torch.stack([w[int(s >= 250000)].double().abs() @ grad[s].double().abs() for s in some])
    ref.close(dxs[some], want, tolerance(want, mag, F, dt))
    for e in range(E):
        at = some[(some >= 250000) == bool(e)]
        want, mag = (f(xs[at].double()).T @ f(grad[at].double()) for f in (lambda x: x, torch.abs))
        ref.close(dw[e], want, tolerance(want, mag, 250000, dt))


def test_empty(sdm, cuda_device):
    dt = torch.bfloat16
    for T, k, E, H, F in ((0, 2, 4, 16, 16), (3, 0, 4, 16, 16), (3, 2, 0, 16, 16), (3, 2, 4, 0, 16),
                          (3, 2, 4, 16, 0)):
        ids = torch.zeros(T, k, dtype=torch.int32, device=cuda_device)
        routes = sdm.ExpertRoutes(ids, E)
        xs, grad = (torch.ones(T * k, n, dtype=dt, device=cuda_device) for n in (H, F))
        w = torch.ones(E, H, F, dtype=dt, device=cuda_device)
        ys = routes.product(xs, w)
        dxs, dw = routes.product_backward(grad, xs, w)
        assert ys.shape == (T * k, F) and dxs.shape == xs.shape and dw.shape == w.shape
        if not (T and k and E and H and F):
            assert not ys.any() and not dxs.any() and not dw.any()


def test_reproducible_and_streams(sdm, cuda_device):
    T, k, E, H, F, dt = 500, 4, 16, 256, 512, torch.bfloat16
    routes = sdm.ExpertRoutes(make_ids(T, k, E, 2).to(cuda_device), E)
    xs, dys = (randn(cuda_device, 1 + i, T * k, n).to(dt) for i, n in enumerate((H, F)))
    w = matrices(cuda_device, 3, E, H, F, dt, "in_out")
    want = [routes.product(xs, w), *routes.product_backward(dys, xs, w)]
    side = [torch.cuda.Stream() for _ in range(3)]
    for s in side:                               # a stream hears of captured waits that gave up before
        try:
            sdm.dynamic_sync(s)
        except sdm.SpmmError:
            pass
    torch.cuda.synchronize()
    got = []
    for s in side:                               # three at once, by argument and as current
        got.append([routes.product(xs, w, stream=s), *routes.product_backward(dys, xs, w, stream=s)])
        with torch.cuda.stream(s):
            got.append([routes.product(xs, w), *routes.product_backward(dys, xs, w)])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    for s in side:
        sdm.dynamic_sync(s)


def test_refusals(sdm, cuda_device):
    dt = torch.bfloat16
    routes = sdm.ExpertRoutes(make_ids(4, 2, 3, 1).to(cuda_device), 3)
    xs = torch.ones(8, 16, dtype=dt, device=cuda_device)
    w = torch.ones(3, 16, 24, dtype=dt, device=cuda_device)
    grad = torch.ones(8, 24, dtype=dt, device=cuda_device)
    routes.product(xs, w)
    flat = torch.ones(3 * 16 * 24 + 8, dtype=dt, device=cuda_device)
    for bad_xs, bad_w, err in (
            (xs[:7], w, ValueError), (xs[:, ::2], w[:, ::2], ValueError), (xs.cpu(), w, ValueError),
            (xs, w[:2], ValueError), (xs, w[:, :8], ValueError), (xs, w.half(), TypeError),
            (xs.half(), w, TypeError), (xs.float(), w.float(), ValueError),
            (xs, w[..., :12], ValueError), (xs, w[..., ::2], ValueError), (xs, w[0], ValueError),
            (xs, flat[1:-7].view(3, 16, 24), ValueError), (xs, w.cpu(), ValueError),
            (xs[:, :12].contiguous(), w[:, :12], ValueError),
            (xs, w[:, :1].expand(3, 16, 24), ValueError), (None, w, TypeError)):
        with pytest.raises(err):
            routes.product(bad_xs, bad_w)
    for bad in (grad[:, :16], grad[:4], grad.half(), grad.t().contiguous().t()):
        with pytest.raises((ValueError, TypeError)):
            routes.product_backward(bad, xs, w)


@pytest.mark.parametrize("stored", ["in_out", "out_in"])
@pytest.mark.parametrize("T,E,H,F,last", [
    (5000, 1, 72, 264, 5000),                    # one expert, parts of unlike lengths
    (4096, 2, 128, 128, 4096),                   # an expert without slots
    (1537, 1, 8, 8, 1537), (2600, 2, 520, 40, 2599), (9000, 3, 136, 296, 700)])
def test_slots_summed_in_parts(sdm, cuda_device, T, E, H, F, last, stored):
    """Few experts with many slots: the matrices' gradient is summed in parts of them, of which
    some may have no slot at all."""
    from sparse_dense_matrix_gb300 import dynamic
    assert dynamic.lib.spmm_routes_product_weights_workspace(T, E, H, F) > 0
    dt = torch.float16
    ids = torch.zeros(T, dtype=torch.int32)
    ids[:last] = E - 1
    routes = sdm.ExpertRoutes(ids[:, None].to(cuda_device), E)
    xs, dys = (randn(cuda_device, 1 + i, T, n).to(dt) for i, n in enumerate((H, F)))
    w = matrices(cuda_device, 3, E, H, F, dt, stored)
    want = expected(routes.offsets, xs, w, dys)
    for _ in range(2):                           # the scratch holds the first call's parts
        for g, (x, tol) in zip(routes.product_backward(dys, xs, w), want[1:]):
            ref.close(g, x, tol)
    sdm.dynamic_sync()
