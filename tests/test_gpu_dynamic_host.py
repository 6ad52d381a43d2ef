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


def test_timeouts_are_told_to_their_stream(sdm, cuda_device):
    """A wait that gave up on one stream: another stream's question does not take the
    answer away. The waits are bounded (2 ms) and nothing else is wrong with the device."""
    from sparse_dense_matrix_gb300 import SpmmError, dynamic
    a, b, c = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.Stream()
    sync, fail = sdm.dynamic_sync, dynamic.lib.spmm_dynamic_check_wait_timeout

    def told(stream):
        try:
            sync(stream)
        except SpmmError as e:
            assert e.name == "SPMM_ERR_TIMEOUT"
            return True
        return False

    for s in (a, b, c):                          # whatever was before
        told(s)
        assert not told(s)
    assert fail(2000, a.cuda_stream) == 0
    a.synchronize()
    assert [told(s) for s in (c, b, a, a, b, c)] == [False, False, True, False, False, False]
    assert fail(2000, a.cuda_stream) == 0 and fail(2000, b.cuda_stream) == 0
    torch.cuda.synchronize()
    assert [told(s) for s in (b, a, c, b, a)] == [True, True, False, False, False]
    # one in a captured graph may have run on any stream
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert fail(2000, torch.cuda.current_stream().cuda_stream) == 0
    assert not told(b)
    with torch.cuda.stream(b):
        graph.replay()
    torch.cuda.synchronize()
    assert [told(s) for s in (a, b, c, a, b, c)] == [True] * 3 + [False] * 3
    told(torch.cuda.current_stream())


@pytest.mark.parametrize("limit", [0, -1, 10 ** 7 + 1])
def test_wait_check_refuses(sdm, cuda_device, limit):
    from sparse_dense_matrix_gb300 import dynamic
    assert dynamic.lib.spmm_dynamic_check_wait_timeout(limit, None) == 1
