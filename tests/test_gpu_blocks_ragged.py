"""Blocks of 128 keys whose sequences end inside the first half of their last block, in
a cache that goes on: the kernels by tile walk such a block as two halves, and nobody
sees a key of the second."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import dynamic_ref as ref  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK, NB, Tq, Hq, Hk = 128, 8, 300, 4, 1


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


def problem(sdm, dev, dtype, D, tail, causal):
    """Sequences of 1 to 7 blocks, the last with `tail` keys, all of them in every list:
    unions of 1 to 7 blocks. What lies past a length is NaN."""
    g = torch.Generator(device=dev).manual_seed(tail * D)
    lengths = [BLOCK * u + tail for u in range(7)]
    B, Tk = len(lengths), BLOCK * NB
    q, grad = (torch.randn(B, Tq, Hq, D, generator=g, device=dev).to(DT[dtype]) for _ in range(2))
    k, v = (torch.randn(B, Tk, Hk, D, generator=g, device=dev).to(DT[dtype]) for _ in range(2))
    for b, n in enumerate(lengths):
        k[b, n:] = v[b, n:] = float("nan")
    blocks = torch.arange(7, dtype=torch.int32, device=dev).expand(B, Tq, Hk, 7).contiguous()
    L = torch.tensor(lengths, dtype=torch.int32, device=dev)
    return sdm.BlockSelection(blocks, BLOCK, Tk, L, causal), q, k, v, grad, L


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tail", [1, 20, 63, 64, 65])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", list(DT))
def test_forward(sdm, cuda_device, dtype, D, tail, causal):
    sel, q, k, v, _, L = problem(sdm, cuda_device, dtype, D, tail, causal)
    want = ref.attend(q, k, v, sel.blocks, BLOCK, L, causal)
    for _ in range(3):
        out, lse = sel.attend(q, k, v)
        ref.close(out, want["out"], want["tol_out"], "out")
        ref.close(lse, want["lse"], want["tol_lse"], "lse")
    sdm.dynamic_sync()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tail", [1, 20, 63, 64, 65])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", list(DT))
def test_gradients(sdm, cuda_device, dtype, D, tail, causal):
    sel, q, k, v, grad, L = problem(sdm, cuda_device, dtype, D, tail, causal)
    want = ref.attend(q, k, v, sel.blocks, BLOCK, L, causal, grad=grad)
    out, lse = sel.attend(q, k, v)
    for _ in range(3):
        for name, got in zip(("dq", "dk", "dv"), sel.backward(grad, q, k, v, out, lse)):
            ref.close(got, want[name], want["tol_" + name], name)
    sdm.dynamic_sync()
