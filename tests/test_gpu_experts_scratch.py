"""The matrices' gradient of few experts with many slots, whose parts go through scratch, in
threads that share a stream, on other streams and in a captured graph."""
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


def told(sdm, stream=None):
    """A stream hears of captured waits that gave up before: it is asked first."""
    try:
        sdm.dynamic_sync(stream)
    except sdm.SpmmError:
        pass


def problem(sdm, dev, seed, T=5000, E=1, H=72, F=264):
    from sparse_dense_matrix_gb300 import dynamic
    assert dynamic.lib.spmm_routes_product_weights_workspace(T, E, H, F) > 0
    ids = torch.arange(T, dtype=torch.int32, device=dev)[:, None] % E
    xs, grad, w = (randn(dev, 3 * seed + i, *s).bfloat16()
                   for i, s in enumerate(((T, H), (T, F), (E, H, F))))
    return sdm.ExpertRoutes(ids.contiguous(), E), grad, xs, w


def test_threads_that_share_a_stream(sdm, cuda_device):
    dev = cuda_device
    work = [problem(sdm, dev, i, E=1 + i % 2) for i in range(4)]
    want = [r.product_backward(*a) for r, *a in work]
    torch.cuda.synchronize()
    told(sdm)
    failed = []

    def thread(i):
        try:
            torch.cuda.set_device(dev)
            r, *a = work[i]
            for _ in range(200):
                # blocks of the scratch's and other sizes, written and given back at once
                for n in (1 << 20, 72 * 264 * 39 * 4, 100):
                    torch.empty(n, dtype=torch.uint8, device=dev).fill_(255)
                got = r.product_backward(*a)
            torch.cuda.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(want[i], got)):
                failed.append("results differ")
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    sdm.dynamic_sync()


def test_streams_and_graph(sdm, cuda_device):
    dev = cuda_device
    r, grad, xs, w = problem(sdm, dev, 7)
    want = r.product_backward(grad, xs, w)
    side = [torch.cuda.Stream() for _ in range(3)]
    for s in side:
        told(sdm, s)
    torch.cuda.synchronize()
    got = []
    for s in side:
        got.append(r.product_backward(grad, xs, w, stream=s))
        with torch.cuda.stream(s):
            got.append(r.product_backward(grad, xs, w))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))
    for s in side:
        sdm.dynamic_sync(s)
    # two graphs, replayed in turn and at once
    graphs, kept = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            kept.append(r.product_backward(grad, xs, w))
    grad.copy_(randn(dev, 50, *grad.shape))
    torch.cuda.synchronize()
    for s, g in zip(side, graphs):
        with torch.cuda.stream(s):
            for _ in range(20):
                g.replay()
    torch.cuda.synchronize()
    want = r.product_backward(grad, xs, w)
    assert all(torch.equal(a, b) for k in kept for a, b in zip(want, k))
    sdm.dynamic_sync()


def test_one_of_many_experts_holds_all_slots(sdm, cuda_device):
    """More than 2^24 slots of one of 160 experts: as many tiles as there are SMs, of which one
    has all the work. It is summed in parts."""
    import dynamic_ref as ref
    from sparse_dense_matrix_gb300 import dynamic
    dev, dt = cuda_device, torch.bfloat16
    T, E, H, F, hot = (1 << 24) + 12345, 160, 8, 16, 77
    assert dynamic.lib.spmm_routes_product_weights_workspace(T, E, H, F) == 2 * E * H * F * 4
    ids = torch.full((T, 1), hot, dtype=torch.int32, device=dev)
    ids[-100:] = 3
    routes = sdm.ExpertRoutes(ids, E)
    xs, grad = (torch.zeros(T, n, dtype=dt, device=dev) for n in (H, F))
    # rows at the parts' ends and beginnings; the others add 0, exactly
    half = (T - 100 + 1) // 2
    some = torch.tensor([0, 99, 100, 101, 63 + 100, 4000000, half + 90, half + 110, half + 170,
                         (1 << 24) - 1, 1 << 24, T - 1], device=dev)
    xs[some], grad[some] = randn(dev, 1, len(some), H).to(dt), randn(dev, 2, len(some), F).to(dt)
    w = randn(dev, 3, E, H, F).to(dt)
    told(sdm)
    dxs, dw = routes.product_backward(grad, xs, w)
    sdm.dynamic_sync()
    for e, at in ((3, some[some < 100]), (hot, some[some >= 100])):
        x, g = xs[at].double(), grad[at].double()
        want, mag = x.T @ g, x.abs().T @ g.abs()
        # as many terms as there are rows, what an instruction may cut off of them, one rounding
        ref.close(dw[e], want, ref.U[dt] * want.abs() + (len(at) + 32) * ref.E32 * mag)
        dw[e] = 0
        want, mag = g @ w[e].double().T, g.abs() @ w[e].double().abs().T
        ref.close(dxs[at], want, ref.U[dt] * want.abs() + (F + 32) * ref.E32 * mag)
    assert not dw.any()
    dxs[some] = 0
    assert not dxs.any()


def test_launches_right_behind_one_another(sdm, cuda_device):
    """Products of pairs and of single CTAs, their gradients and the attention's tile kernels in
    turn on the same SMs: each begins with barriers of its own in the shared memory that the
    one before has just left."""
    dev, dt = cuda_device, torch.bfloat16
    E, H, F = 8, 256, 264
    ids = torch.arange(2000, dtype=torch.int32, device=dev)[:, None] * 5 % E
    many, few = sdm.ExpertRoutes(ids.contiguous(), E), sdm.ExpertRoutes(ids[:40].contiguous(), E)
    xs, grad, w = (randn(dev, i, *s).to(dt)
                   for i, s in enumerate(((2000, H), (2000, F), (E, H, F))))
    q, k, v = (randn(dev, 3 + i, 1, 300, n, 64).to(dt) for i, n in enumerate((8, 2, 2)))
    sel = sdm.select_blocks(q, sdm.block_means(k, 64), 3, 64, 300)

    def step():
        return [many.product(xs, w), sel.attend(q, k, v)[0], few.product(xs[:40], w),
                *many.product_backward(grad, xs, w), sel.attend(q, k, v)[0],
                *few.product_backward(grad[:40], xs[:40], w)]

    told(sdm)
    want = step()
    for _ in range(100):
        got = step()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    sdm.dynamic_sync()
