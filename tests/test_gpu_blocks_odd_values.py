"""Values that are not finite, further: rows whose scores are all -infinity, and the time
of a step whose gradients are all NaN."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


@pytest.mark.parametrize("T", [64, 400])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", list(DT))
def test_rows_whose_scores_are_all_minus_infinity(sdm, cuda_device, dtype, D, T):
    """Their weights are 0: they add nothing to dk and dv, also where another row's
    gradient is NaN and the keys that do not see it are summed on their own."""
    block, Hq = 64, 4
    q, k, v, grad = (randn(cuda_device, i, 1, T, H, D).to(DT[dtype])
                     for i, H in ((0, Hq), (1, 1), (2, 1), (3, Hq)))
    q[..., 0] = 1
    k[0, :11, 0, 0] = -math.inf              # rows 0 to 10 see nothing else
    own = torch.arange(T, device=cuda_device, dtype=torch.int32) // block
    sel = sdm.BlockSelection(own[None, :, None, None].expand(1, T, 1, 1).contiguous(), block, T)
    out, lse = sel.attend(q, k, v)
    assert (lse[0, :11] == -math.inf).all() and (out[0, :11] == 0).all()
    _, dk, dv = sel.backward(grad, q, k, v, out, lse)
    grad[0, 3] = math.nan                    # seen by keys 0 to 3 only
    _, dk2, dv2 = sel.backward(grad, q, k, v, out, lse)
    assert torch.isfinite(dk).all() and torch.isfinite(dv).all()
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[q.dtype]
    for a, b in ((dk, dk2), (dv, dv2)):      # alone: rounded once, from unrounded weights
        assert torch.isfinite(b[0, 4:]).all()
        assert (a[0, 4:] - b[0, 4:]).abs().max() <= 4 * u * a.abs().max() + 32 * u
    sdm.dynamic_sync()


def timed(f):
    """ms, the best of seven: the launches are the host's, which may be held up."""
    best = math.inf
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("dtype,D,block", [("bf16", 128, 64), ("bf16", 64, 64), ("fp16", 128, 64),
                                           ("fp16", 64, 16)])
@pytest.mark.parametrize("what", ["grad", "v", "q"])
def test_time_of_a_step_that_is_all_nan(sdm, cuda_device, dtype, D, block, what):
    """A step whose loss overflowed gives NaN everywhere in a small multiple of its time: the
    rows that are computed again alone stop once nothing of them can change. (Without
    that it was a multiple of hundreds.)"""
    B, T, Hq, Hk, n = 1, 2048, 16, 2, 1024 // block
    q, k, v, grad = (randn(cuda_device, i, B, T, H, D).to(DT[dtype])
                     for i, H in ((0, Hq), (1, Hk), (2, Hk), (3, Hq)))
    sel = sdm.select_blocks(q, sdm.block_means(k, block), n, block, T)

    def step():
        out, lse = sel.attend(q, k, v)
        return (out, *sel.backward(grad, q, k, v, out, lse))

    clean = timed(step)
    {"grad": grad, "v": v, "q": q}[what].fill_(math.nan)
    odd = timed(step)
    print(f"clean {clean:.3f} ms, NaN {odd:.3f} ms")
    out, dq, dk, dv = step()
    if what != "grad":
        assert torch.isnan(out).all()
    assert torch.isnan(dq).all() and torch.isnan(dk).all()
    assert what == "v" or torch.isnan(dv).all()
    assert odd <= 12 * clean
    sdm.dynamic_sync()
