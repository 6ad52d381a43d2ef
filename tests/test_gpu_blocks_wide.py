"""More (sequence, kv head) pairs than one launch dimension holds: whatever the forward
takes, the means, the selection and the gradient take."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import dynamic_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


@pytest.mark.parametrize("B,Hk,Tq", [(65536 + 9, 1, 2), (33000, 2, 24), (65536 + 9, 1, 25)])
def test_many_sequences(sdm, cuda_device, B, Hk, Tq):
    Tk, D, block, n = 40, 64, 16, 2
    g = torch.Generator(device=cuda_device).manual_seed(Tq)
    rnd = lambda T: torch.randn(B, T, Hk, D, generator=g, device=cuda_device)  # noqa: E731
    q, k = ((rnd(T) * 8).round_().mul_(0.125).half() for T in (Tq, Tk))
    v, grad = rnd(Tk).half(), rnd(Tq).half()
    m = sdm.block_means(k, block)
    sel = sdm.select_blocks(q, m, n, block, Tk)
    out, lse = sel.attend(q, k, v)
    got = dict(zip(("dq", "dk", "dv"), sel.backward(grad, q, k, v, out, lse)), out=out, lse=lse)
    some = [0, 1, 32767, 32768, B - 1] + ([65535, 65536] if B > 65536 else [])
    ref.close(m[some], ref.means(k[some], block, None),
              2 * block * ref.E32 * k.abs().max().double())
    lists, _ = ref.select(q[some], m[some], n, block, Tk, None, True)
    assert torch.equal(sel.blocks[some].cpu(), lists)
    want = ref.attend(q[some], k[some], v[some], sel.blocks[some], block, None, True, grad=grad[some])
    for name in got:
        ref.close(got[name][some], want[name], want["tol_" + name], name)
    sdm.dynamic_sync()
