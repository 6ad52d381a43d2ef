"""Selection for prompts whose scores do not fit the scratch at once."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,T,Hk,block,n", [(1, 40011, 4, 16, 9), (2, 30000, 3, 16, 40),
                                            (1, 100003, 2, 64, 16)])
def test_strips_of_queries(sdm, cuda_device, B, T, Hk, block, n, causal):
    """The lists of the queries from a to b of a prompt of T tokens are those of a chunk of
    these queries over the same keys."""
    D, Hq = 64, 2 * Hk
    g = torch.Generator(device=cuda_device).manual_seed(T)
    q, k = ((torch.randn(B, T, H, D, generator=g, device=cuda_device) * 8).round_().mul_(0.125)
            .bfloat16() for H in (Hq, Hk))
    m = sdm.block_means(k, block)
    assert B * T * Hk * m.shape[1] * 4 > 1 << 30           # else one strip holds it
    whole = sdm.select_blocks(q, m, n, block, T, causal=causal).blocks
    for a, b in ((0, 100), (T // 2, T // 2 + 1), (22220, 22420), (26780, 26900), (T - 130, T - 3),
                 (T - 1, T), (0, T // 3), (T // 3, T)):
        # a chunk that ends at position b - 1; the other keys lie after it
        L = torch.full((B,), b if causal else T, dtype=torch.int32, device=cuda_device)
        part = sdm.select_blocks(q[:, a:b], m, n, block, T, L, causal).blocks
        assert torch.equal(part, whole[:, a:b]), (a, b)
