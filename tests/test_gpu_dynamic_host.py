"""The run-time patterns' host side on the GPU: calls from several threads."""
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sdm(cuda_device):
    import sparse_dense_matrix_gb300 as m
    return m


def test_sorts_of_two_threads(sdm, cuda_device):
    """Both numbers of experts need more shared memory than a kernel has by default, and
    different amounts of it."""
    ids = torch.zeros(8, 2, dtype=torch.int32, device=cuda_device)
    failed = []

    def sort(E):
        torch.cuda.set_device(cuda_device)
        try:
            for _ in range(4000):
                sdm.ExpertRoutes(ids, E)
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)

    threads = [threading.Thread(target=sort, args=(E,)) for E in (2048, 800, 2048, 800)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
