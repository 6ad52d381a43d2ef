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
