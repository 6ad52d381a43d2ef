"""Copies of routes, rotations and selections, and what a file gives back, are used after the
originals are gone and their memory has been given out again."""
import copy
import io

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


def written(x):
    f = io.BytesIO()
    torch.save(x, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


def overwrite(dev):
    """What the allocator has of free small blocks is filled with other numbers."""
    for n in (16, 64, 256, 1024, 4096) * 50:
        torch.full((n,), -1, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, written])
def test_copied_routes(sdm, cuda_device, how):
    dev = cuda_device
    ids = (torch.arange(200, dtype=torch.int32, device=dev) * 7 % 5).view(100, 2)
    x, w = randn(dev, 1, 100, 64).bfloat16(), randn(dev, 2, 5, 64, 72).bfloat16()
    routes = sdm.ExpertRoutes(ids, 5)
    want = [routes.dispatch(x), routes.product(routes.dispatch(x), w)]
    other = how(routes)
    del routes
    torch.cuda.synchronize()
    overwrite(dev)
    xs = other.dispatch(x)
    assert torch.equal(xs, want[0]) and torch.equal(other.product(xs, w), want[1])


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, written])
def test_copied_rotation(sdm, cuda_device, how):
    dev = cuda_device
    rot, q = sdm.HeadRotation(128, device=dev), randn(dev, 1, 2, 50, 4, 128)
    want = rot.rotate(q)[0]
    other = how(rot)
    del rot
    torch.cuda.synchronize()
    overwrite(dev)
    assert torch.equal(other.rotate(q)[0], want)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, written])
@pytest.mark.parametrize("lengths", [False, True])
def test_copied_selection(sdm, cuda_device, lengths, how):
    dev = cuda_device
    q, k, v = (randn(dev, i, 2, 70, h, 64).bfloat16() for i, h in enumerate((4, 2, 2)))
    L = torch.tensor([70, 41], dtype=torch.int32, device=dev) if lengths else None
    sel = sdm.select_blocks(q, sdm.block_means(k, 16, L), 3, 16, 70, L)
    want = sel.attend(q, k, v)
    given = sdm.BlockSelection(sel.blocks.clone(), 16, 70, L)
    others = [how(sel), how(given)]
    del sel, given
    torch.cuda.synchronize()
    overwrite(dev)
    for other in others:
        assert all(torch.equal(a, b) for a, b in zip(other.attend(q, k, v), want))


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy])
def test_copies_on_another_stream_keep_their_memory(sdm, cuda_device, how):
    """A copy made and used on another stream than the original, whose tensors it may share."""
    dev, side = cuda_device, torch.cuda.Stream()
    q = randn(dev, 1, 1, 4096, 8, 128)
    rot = sdm.HeadRotation(128, device=dev)
    want = rot.rotate(q)[0]
    del rot
    for _ in range(2):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        rot = sdm.HeadRotation(128, device=dev)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = how(rot)
            torch.cuda._sleep(200_000_000)       # 0.1 s
            got = other.rotate(q)[0]
        ptr, nbytes = other.turns.data_ptr(), other.turns.numel() * 8
        del rot, other
        keep = [torch.empty(nbytes, dtype=torch.uint8, device=dev) for _ in range(20)]
        assert not side.query(), "the side stream is done already: nothing was tested"
        assert not any(t.data_ptr() < ptr + nbytes and ptr < t.data_ptr() + nbytes for t in keep)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
