"""What a selection keeps (the lengths that it was made for), and strides that mean nothing."""
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


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Tq,Tk", [(1, 300), (40, 300), (100, 20000)])
@pytest.mark.parametrize("made", ["selected", "given"])
def test_lengths_updated_in_place(sdm, cuda_device, made, Tq, Tk, causal):
    """A decode loop adds to its lengths in place: a selection made before goes on with
    the lengths that it was made for."""
    B, Hq, Hk, D, block, n = 3, 4, 2, 64, 16, 5
    q, grad = randn(cuda_device, 1, B, Tq, Hq, D).half(), randn(cuda_device, 2, B, Tq, Hq, D).half()
    k, v = randn(cuda_device, 3, B, Tk, Hk, D).half(), randn(cuda_device, 4, B, Tk, Hk, D).half()
    L = torch.tensor([100, 0, 257], dtype=torch.int32, device=cuda_device)
    sel = sdm.select_blocks(q, sdm.block_means(k, block, L), n, block, Tk, L, causal)
    if made == "given":
        sel = sdm.BlockSelection(sel.blocks, block, Tk, L, causal)
    out, lse = sel.attend(q, k, v)
    want = (out, lse, *sel.backward(grad, q, k, v, out, lse))
    before = L.clone()
    L += 17
    out, lse = sel.attend(q, k, v)
    for a, b in zip(want, (out, lse, *sel.backward(grad, q, k, v, out, lse))):
        assert torch.equal(a, b)
    assert torch.equal(sel.lengths, before)
    sdm.dynamic_sync()


def test_lengths_without_queries(sdm, cuda_device):
    L = torch.tensor([5, 9], dtype=torch.int32, device=cuda_device)
    q, k = (randn(cuda_device, 1, 2, T, 2, 64).half() for T in (0, 12))
    sel = sdm.select_blocks(q, sdm.block_means(k, 16, L), 2, 16, 12, L)
    before = L.clone()
    L += 1
    assert torch.equal(sel.lengths, before) and sel.blocks.shape == (2, 0, 2, 2)
    assert sdm.select_blocks(q, sdm.block_means(k, 16), 2, 16, 12).lengths is None


def test_strides_of_dimensions_of_one(sdm, cuda_device):
    """They mean nothing, and torch gives them any value."""
    D = 64
    for dt in (torch.bfloat16, torch.float16):
        q, k, v, g = (randn(cuda_device, i, D, 1).to(dt).t()[None, None] for i in range(4))
        assert q.shape == (1, 1, 1, D) and q.stride(2) == 1
        sel = sdm.select_blocks(q, sdm.block_means(k, 16), 1, 16, 1)
        out, lse = sel.attend(q, k, v)
        assert torch.equal(out, v.contiguous())
        dq, dk, dv = sel.backward(g, q, k, v, out, lse)
        assert torch.equal(dv, g.contiguous())
    # one head of many queries, its stride an odd number
    T = 300
    q, k, v = (torch.as_strided(randn(cuda_device, i, T * D).half(), (1, T, 1, D), (1, D, 3, 1))
               for i in range(3))
    def run(q, k, v):
        sel = sdm.select_blocks(q, sdm.block_means(k, 32), 4, 32, T)
        out, lse = sel.attend(q, k, v)
        return (sel.blocks, out, lse, *sel.backward(q, q, k, v, out, lse))
    want = run(*(x.contiguous().clone(memory_format=torch.contiguous_format).view(1, T, 1, D)
                 for x in (q, k, v)))
    assert all(torch.equal(a, b) for a, b in zip(want, run(q, k, v)))
