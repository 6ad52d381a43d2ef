"""Tensors used on another stream than their own keep their memory until it is done."""
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


def reused(ptr, nbytes, dev):
    """Whether tensors made now on the current stream take bytes of [ptr, ptr + nbytes)."""
    keep = [torch.empty(nbytes, dtype=torch.uint8, device=dev) for _ in range(20)]
    return any(t.data_ptr() < ptr + nbytes and ptr < t.data_ptr() + nbytes for t in keep)


def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)          # 0.1 s


def test_routes_on_another_stream_keep_their_memory(sdm, cuda_device):
    T, k, E, H = 1 << 19, 4, 8, 16
    ids = torch.zeros(T, k, dtype=torch.int32, device=cuda_device)
    x = torch.ones(T, H, device=cuda_device)
    w = torch.ones(T, k, device=cuda_device)
    side = torch.cuda.Stream()
    for how in ("argument", "current"):
        for call in ("dispatch", "combine", "combine_backward"):
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            routes = sdm.ExpertRoutes(ids, E)
            xs = routes.dispatch(x)
            torch.cuda.synchronize()
            ptr, nbytes = routes.slots.data_ptr(), routes.slots.numel() * 4
            busy(side)
            args = {"dispatch": (x,), "combine": (xs, w), "combine_backward": (x, xs, w)}[call]
            if how == "argument":
                got = getattr(routes, call)(*args, stream=side)
            else:
                with torch.cuda.stream(side):
                    got = getattr(routes, call)(*args)
            del routes, xs
            args = None
            assert not side.query(), "the side stream is done already: nothing was tested"
            assert not reused(ptr, nbytes, cuda_device), (how, call)
            torch.cuda.synchronize()
            del got


def test_inputs_on_a_given_stream_keep_their_memory(sdm, cuda_device):
    T, k, E, H = 1 << 16, 2, 8, 64
    ids = torch.zeros(T, k, dtype=torch.int32, device=cuda_device)
    routes = sdm.ExpertRoutes(ids, E)
    side = torch.cuda.Stream()
    x = torch.ones(T, H, device=cuda_device)
    torch.cuda.synchronize()
    ptr, nbytes = x.data_ptr(), x.numel() * 4
    busy(side)
    got = routes.dispatch(x, stream=side)
    del x
    assert not side.query() and not reused(ptr, nbytes, cuda_device)
    torch.cuda.synchronize()
    assert (got == 1).all()
    x = torch.zeros(T, k, dtype=torch.int32, device=cuda_device)
    torch.cuda.synchronize()
    ptr, nbytes = x.data_ptr(), x.numel() * 4
    busy(side)
    sdm.ExpertRoutes(x, E, stream=side)
    del x
    assert not side.query() and not reused(ptr, nbytes, cuda_device)
    torch.cuda.synchronize()


def test_selections_on_another_stream_keep_their_memory(sdm, cuda_device):
    B, T, Hq, Hk, D, block, n = 1, 8192, 2, 2, 64, 16, 32
    q, k, v, g = (randn(cuda_device, i, B, T, H, D).half()
                  for i, H in ((0, Hq), (1, Hk), (2, Hk), (3, Hq)))
    L = torch.full((B,), T, dtype=torch.int32, device=cuda_device)
    m = sdm.block_means(k, block, L)
    side = torch.cuda.Stream()
    for how in ("argument", "current"):
        for call in ("attend", "backward"):
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            sel = sdm.select_blocks(q, m, n, block, T, L)
            out, lse = sel.attend(q, k, v)
            torch.cuda.synchronize()
            ptr, nbytes = sel.blocks.data_ptr(), sel.blocks.numel() * 4
            args = (q, k, v) if call == "attend" else (g, q, k, v, out, lse)
            busy(side)
            if how == "argument":
                got = getattr(sel, call)(*args, stream=side)
            else:
                with torch.cuda.stream(side):
                    got = getattr(sel, call)(*args)
            del sel
            assert not side.query(), "the side stream is done already: nothing was tested"
            assert not reused(ptr, nbytes, cuda_device), (how, call)
            torch.cuda.synchronize()
            del got
    # and the inputs of a call on a given stream
    for call in ("means", "select", "attend", "backward"):
        torch.cuda.synchronize()
        sel = sdm.select_blocks(q, m, n, block, T, L)
        out, lse = sel.attend(q, k, v)
        mine = {"means": k, "select": q, "attend": v, "backward": out}[call].clone()
        torch.cuda.synchronize()
        ptr, nbytes = mine.data_ptr(), mine.numel() * 2
        busy(side)
        got = {"means": lambda x: sdm.block_means(x, block, L, stream=side),
               "select": lambda x: sdm.select_blocks(x, m, n, block, T, L, stream=side),
               "attend": lambda x: sel.attend(q, k, x, stream=side),
               "backward": lambda x: sel.backward(g, q, k, v, x, lse, stream=side)}[call](mine)
        del mine
        assert not side.query() and not reused(ptr, nbytes, cuda_device), call
        torch.cuda.synchronize()
        del got, sel
    sdm.dynamic_sync()


def test_made_outside_and_captured(sdm, cuda_device):
    """Routes and selections made on another stream before a capture, used in it and
    dropped when the graph is done: its results are those of the calls."""
    B, T, H, block, n = 1, 600, 2, 64, 4
    q, k, v = (randn(cuda_device, i, B, T, H, 128).bfloat16() for i in range(3))
    sel = sdm.select_blocks(q, sdm.block_means(k, block), n, block, T,
                            torch.tensor([580], dtype=torch.int32, device=cuda_device))
    routes = sdm.ExpertRoutes(torch.arange(T, dtype=torch.int32, device=cuda_device)[:, None] % 7, 7)
    x = randn(cuda_device, 5, T, 64)
    out, lse = sel.attend(q, k, v)
    want = (out, lse, *sel.backward(q, q, k, v, out, lse), routes.dispatch(x))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = sel.attend(q, k, v)
        got = (out, lse, *sel.backward(q, q, k, v, out, lse), routes.dispatch(x))
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    torch.empty(1 << 20, device=cuda_device)             # the allocator is whole
    del sel, routes
    torch.cuda.empty_cache()
    assert torch.ones(8, device=cuda_device).sum() == 8
