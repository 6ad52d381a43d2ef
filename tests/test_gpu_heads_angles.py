"""Small angles: the sines of the slow pairs near position 0 are as exact, of themselves, as
any other value, and so is what an fp32 call makes of them."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import dynamic_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("base,scaling", [
    (1e4, None), (5e5, None), (5e5, {"kind": "linear", "factor": 32.0}),
    (1e7, {"kind": "base", "factor": 8.0})])
def test_sines_near_position_0(sdm, cuda_device, base, scaling, layout):
    """A head (1, 0) of each pair becomes (cos, sin), and its gradient (cos, -sin)."""
    D, dev = 128, cuda_device
    rot = sdm.HeadRotation(D, layout=layout, base=base, scaling=scaling, device=dev)
    at = [1, -1, 2, -2, 5, -7, 0]
    q = torch.zeros(1, len(at), 1, D, device=dev)
    first, second = ((slice(0, D // 2), slice(D // 2, D)) if layout == "half"
                     else (slice(0, D, 2), slice(1, D, 2)))
    q[..., first] = 1
    pos = torch.tensor(at, dtype=torch.int32, device=dev)
    got = rot.rotate(q, positions=pos)[0][0, :, 0, second].double().cpu()
    back = rot.rotate_backward(q, None, positions=pos)[0][0, :, 0, second].double().cpu()
    for t, p in enumerate(at):
        for i, f in enumerate(rot.frequencies):
            want = math.sin(p * f)
            # of itself: 5 E for the angle (3 of its own, which the sine of a small angle
            # follows whole) and the series' terms (4 of the second one, which only near a
            # quarter turn is more than half of the sum, and 1 left out there), 1 for the last
            # rounding. Besides, the frequency in turns is rounded to 2^-64 of one, and its
            # division by 2 pi, the product p f here and their host's functions to 2^-53 each
            tol = 6 * ref.E32 * abs(want) + abs(p) * (math.tau * 2.0 ** -65 + 3 * 2.0 ** -52 * f)
            assert abs(got[t, i].item() - want) <= tol, (p, i)
            assert abs(back[t, i].item() + want) <= tol, (p, i)
