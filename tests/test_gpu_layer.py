"""The experts' products and the heads' norm and rotation as a layer uses them: the example's
whole step as a captured graph, memory of tensors used on another stream, calls of several
threads, and the state that calls leave behind."""
import os
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


def test_layer_step_captured(sdm, cuda_device):
    """Nothing in the layer waits for the device, so that a whole training step and a token
    can be captured; their replays on other inputs give the calls' results."""
    from sparse_layer import SparseLayer
    layer = SparseLayer(device=cuda_device)
    B, T, H = 2, 100, layer.hidden
    x, grad = (randn(cuda_device, i, B, T, H).bfloat16() for i in (1, 2))
    ck, cv = (torch.zeros(B, T + 1, layer.kv_heads, layer.dim, dtype=x.dtype, device=cuda_device)
              for _ in range(2))
    L = torch.full((B,), T, dtype=torch.int32, device=cuda_device)

    def step():
        y, saved = layer.prompt(x)
        grads = layer.prompt_backward(grad, saved)
        ck[:, :T], cv[:, :T] = saved[1], saved[2]
        L.fill_(T)
        means = sdm.block_means(ck, layer.block, L)
        one = layer.token(x[:, :1], ck, cv, means, L)
        return [y, *grads.values(), one, means, ck.clone(), cv.clone(), L.clone()]

    for _ in range(2):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6):
        x.copy_(randn(cuda_device, seed, B, T, H))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(torch.isfinite(t).all() for t in got)
    sdm.dynamic_sync()


def reused(ptr, nbytes, dev):
    """Whether tensors made now on the current stream take bytes of [ptr, ptr + nbytes)."""
    keep = [torch.empty(nbytes, dtype=torch.uint8, device=dev) for _ in range(20)]
    return any(t.data_ptr() < ptr + nbytes and ptr < t.data_ptr() + nbytes for t in keep)


def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)           # 0.1 s


def test_inputs_on_another_stream_keep_their_memory(sdm, cuda_device):
    dev, side = cuda_device, torch.cuda.Stream()
    T, k, E, H, F = 4096, 2, 8, 512, 512
    ids = torch.arange(T * k, dtype=torch.int32, device=dev).view(T, k) % E
    routes = sdm.ExpertRoutes(ids, E)
    xs, w, grad = (randn(dev, i, *s).bfloat16()
                   for i, s in enumerate(((T * k, H), (E, H, F), (T * k, F))))
    rot = sdm.HeadRotation(128, device=dev)
    q, kk, v = (randn(dev, 3 + i, 1, 4096, 8, 128).bfloat16() for i in range(3))
    ck, cv = (torch.zeros(1, 4096, 8, 128, dtype=q.dtype, device=dev) for _ in range(2))
    L = torch.full((1,), 4096, dtype=torch.int32, device=dev)
    wt = torch.ones(128, device=dev)
    calls = {
        "product xs": (xs, lambda t: routes.product(t, w, stream=side)),
        "product w": (w, lambda t: routes.product(xs, t, stream=side)),
        "gradient grad": (grad, lambda t: routes.product_backward(t, xs, w, stream=side)),
        "gradient xs": (xs, lambda t: routes.product_backward(grad, t, w, stream=side)),
        "rotate q": (q, lambda t: rot.rotate(t, kk, q_weight=wt, stream=side)),
        "rotate k": (kk, lambda t: rot.rotate(q, t, stream=side)),
        "append v": (v, lambda t: rot.append(q, kk, t, ck, cv, L, stream=side)),
        "append cache": (ck, lambda t: rot.append(q, kk, v, t, cv, L, stream=side)),
        "backward grad": (q, lambda t: rot.rotate_backward(t, kk, stream=side)),
        "backward q": (q, lambda t: rot.rotate_backward(q, kk, t, q_weight=wt, stream=side))}
    for name, (t, call) in calls.items():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        mine = t.clone()
        torch.cuda.synchronize()
        ptr, nbytes = mine.data_ptr(), mine.numel() * mine.element_size()
        busy(side)
        got = call(mine)
        del mine
        assert not side.query(), "the side stream is done already: nothing was tested"
        assert not reused(ptr, nbytes, dev), name
        torch.cuda.synchronize()
        del got
    # and what routes and a rotation hold themselves
    for how in ("argument", "current"):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        routes = sdm.ExpertRoutes(ids, E)
        torch.cuda.synchronize()
        ptr, nbytes = routes.offsets.data_ptr(), routes.offsets.numel() * 4
        busy(side)
        if how == "argument":
            got = routes.product(xs, w, stream=side)
        else:
            with torch.cuda.stream(side):
                got = routes.product(xs, w)
        del routes
        assert not side.query() and not reused(ptr, nbytes, dev), how
        torch.cuda.synchronize()
        rot = sdm.HeadRotation(128, device=dev)
        torch.cuda.synchronize()
        ptr, nbytes = rot.turns.data_ptr(), rot.turns.numel() * 8
        busy(side)
        if how == "argument":
            got = rot.rotate(q, stream=side)
        else:
            with torch.cuda.stream(side):
                got = rot.rotate(q)
        del rot
        assert not side.query() and not reused(ptr, nbytes, dev), how
        torch.cuda.synchronize()
        del got


def test_calls_of_several_threads(sdm, cuda_device):
    """Threads on streams of their own, with numbers of experts that want different amounts
    of shared memory, and one rotation that all of them use."""
    dev = cuda_device
    rot = sdm.HeadRotation(64, device=dev)
    sizes = [(3, 64, 64), (2048, 16, 24), (700, 32, 40), (16, 256, 264)]
    work = []
    for i, (E, H, F) in enumerate(sizes):
        ids = (torch.arange(600, dtype=torch.int32, device=dev) * 7 % E)[:, None].contiguous()
        xs, w = randn(dev, i, 600, H).bfloat16(), randn(dev, 9 + i, E, H, F).bfloat16()
        grad, q = randn(dev, 20 + i, 600, F).bfloat16(), randn(dev, 30 + i, 2, 50 + i, 4, 64)
        L = torch.tensor([50, 70], dtype=torch.int32, device=dev)

        def run(ids=ids, E=E, xs=xs, w=w, grad=grad, q=q, L=L):
            r = sdm.ExpertRoutes(ids, E)
            return [r.product(xs, w), *r.product_backward(grad, xs, w),
                    rot.rotate(q, lengths=L)[0]]

        work.append((run, run()))
    torch.cuda.synchronize()
    failed = []

    def thread(run, want):
        try:
            torch.cuda.set_device(dev)
            s = torch.cuda.Stream()
            try:                                 # captured waits that gave up before, elsewhere
                sdm.dynamic_sync(s)
            except sdm.SpmmError:
                pass
            with torch.cuda.stream(s):
                for _ in range(150):
                    got = run()
                s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(want, got)):
                failed.append("results differ")
            sdm.dynamic_sync(s)
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)

    threads = [threading.Thread(target=thread, args=a) for a in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_outputs_are_written_whole(sdm, cuda_device):
    """Every element of a result is written, on memory that held NaN, and nothing around it."""
    from sparse_dense_matrix_gb300 import dynamic
    dev, dt = cuda_device, torch.bfloat16
    T, k, E, H, F = 37, 3, 5, 72, 136
    ids = torch.randint(-1, E, (T, k), generator=torch.Generator().manual_seed(1)).to(
        dev, torch.int32)
    routes = sdm.ExpertRoutes(ids, E)
    P, stream = T * k, torch.cuda.current_stream().cuda_stream
    xs, w, grad = (randn(dev, i, *s).to(dt) for i, s in enumerate(((P, H), (E, H, F), (P, F))))
    want = [routes.product(xs, w), *routes.product_backward(grad, xs, w)]
    off = routes.offsets.data_ptr()

    def guarded(n):
        room = torch.full((n + 512,), float("nan"), dtype=dt, device=dev)
        return room, room[256:256 + n]

    for name, n in (("ys", P * F), ("dw", E * H * F), ("dw out_in", E * H * F)):
        room, out = guarded(n)
        if name == "ys":
            st = dynamic.lib.spmm_routes_product(1, xs.data_ptr(), w.data_ptr(), H * F, F, 1, off, P,
                                                 E, H, F, out.data_ptr(), stream)
            ref = want[0]
        else:
            sh, sf = (F, 1) if name == "dw" else (1, H)
            st = dynamic.lib.spmm_routes_product_weights(1, xs.data_ptr(), grad.data_ptr(), off, P, E,
                                                         H, F, out.data_ptr(), H * F, sh, sf, None, 0,
                                                         stream)
            ref = want[2] if name == "dw" else want[2].transpose(1, 2).contiguous()
        assert st == 0
        torch.cuda.synchronize()
        assert torch.equal(out, ref.reshape(-1)), name
        room[256:256 + n] = float("nan")
        assert torch.isnan(room).all(), name


def test_bad_offsets_stay_in_bounds(sdm, cuda_device):
    """Offsets that no sort makes (below zero, past the slots, falling) leave the call within its
    tensors: they are clamped, and a first slot below the one before it counts as that."""
    from sparse_dense_matrix_gb300 import dynamic
    dev, dt = cuda_device, torch.float16
    P, E, H, F = 50, 4, 64, 64
    stream = torch.cuda.current_stream().cuda_stream
    xs, w, grad = (randn(dev, i, *s).to(dt) for i, s in enumerate(((P, H), (E, H, F), (P, F))))
    for bad, clamped in (([-5, 10, 7, 90, 2 ** 31 - 1], [0, 10, 10, 50, 50]),
                         ([0, 60, 20, -2 ** 31, 30], [0, 50, 50, 50, 50]),
                         ([20, 30, 40, 45, 48], [20, 30, 40, 45, 48])):
        offsets = torch.tensor(bad, dtype=torch.int32, device=dev)
        ys = torch.full((P, F), float("nan"), dtype=dt, device=dev)
        dw = torch.full((E, H, F), float("nan"), dtype=dt, device=dev)
        L = dynamic.lib
        assert L.spmm_routes_product(2, xs.data_ptr(), w.data_ptr(), H * F, F, 1, offsets.data_ptr(),
                                     P, E, H, F, ys.data_ptr(), stream) == 0
        assert L.spmm_routes_product_weights(2, xs.data_ptr(), grad.data_ptr(), offsets.data_ptr(), P,
                                             E, H, F, dw.data_ptr(), H * F, F, 1, None, 0, stream) == 0
        sdm.dynamic_sync()
        for e in range(E):
            rows = slice(clamped[e], clamped[e + 1])
            # sums of 64 (or up to 50) products: 2^-11 of the rounding and 96 x 2^-24 of terms up to 25
            assert torch.allclose(ys[rows].double(), xs[rows].double() @ w[e].double(), rtol=2.0 ** -11,
                                  atol=96 * 2.0 ** -24 * 64 * 25)
            assert torch.allclose(dw[e].double(), xs[rows].double().T @ grad[rows].double(),
                                  rtol=2.0 ** -11, atol=96 * 2.0 ** -24 * 64 * 25)
        assert not ys[clamped[-1]:].any()
