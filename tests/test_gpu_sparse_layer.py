"""The example layer: its training step is finite, and single tokens over a cache
give the prompt's outputs. (bf16 throughout: the products of one token and of a
whole prompt round differently, a few units of 2^-8 of the largest values. A token
whose router or block scores nearly tie may choose otherwise; the median over the
compared tokens is held to the rounding.)"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("T", [1, 9, 200])
def test_layer(cuda_device, T):
    import sparse_dense_matrix_gb300 as sdm
    from sparse_layer import SparseLayer
    torch.manual_seed(1)
    layer = SparseLayer(device=cuda_device)
    x = torch.randn(3, T, layer.hidden, device=cuda_device).bfloat16()
    y, saved = layer.prompt(x)
    grads = layer.prompt_backward(torch.randn_like(y), saved)
    assert all(torch.isfinite(g).all() for g in grads.values())
    k, v = torch.zeros_like(saved[1]), torch.zeros_like(saved[2])
    lengths = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    means = sdm.block_means(k, layer.block, lengths)
    diffs = []
    for t in range(T):
        one = layer.token(x[:, t:t + 1], k, v, means, lengths)
        diffs.append((one[:, 0].float() - y[:, t].float()).abs().amax(-1))
    scale = y.float().abs().max().item()
    assert torch.cat(diffs).median().item() <= 8 * 2.0 ** -8 * scale
    sdm.dynamic_sync()
