"""The binding's host side without a GPU: devices of streams, scratch, and the package
without torch."""
import os
import subprocess
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sync_asks_the_streams_device(monkeypatch):
    import sparse_dense_matrix_gb300.dynamic as m
    current, asked = [0], []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(m, "_current_device", lambda: current[0])
    monkeypatch.setattr(m, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(m.torch.cuda, "device", Device)
    monkeypatch.setattr(m, "lib", types.SimpleNamespace(
        spmm_dynamic_sync=lambda handle: asked.append((current[0], handle)) or 0))
    for index in (0, 1):
        m.dynamic_sync(types.SimpleNamespace(device=types.SimpleNamespace(index=index),
                                             cuda_stream=7 + index))
    m.dynamic_sync()
    assert asked == [(0, 7), (1, 8), (0, 100)] and current == [0]


def test_selection_scratch_is_bounded():
    """The scores of a prompt grow with the square of its length; the scratch does not."""
    import sparse_dense_matrix_gb300.dynamic as m

    def need(B, Tq, Tk, Hk, block):
        return m.lib.spmm_blocks_select_workspace(
            m._Shape(B, Tq, Tk, 8 * Hk, Hk, 128, block, 16, 1, 1, 1.0, None))

    for block in (16, 64):
        for T in (1 << 15, 1 << 17, 1 << 20):
            one = 8 * (T // block) * 4                       # the scores of one query
            assert one <= need(1, T, T, 8, block) <= max(1 << 30, 64 * one)
    assert need(1, 8192, 8192, 4, 64) == 8192 * 4 * 128 * 4  # a whole prompt that fits


NO_TORCH = {
    "absent": """
import importlib.abc, sys
class NoTorch(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path, target=None):
        if name.partition(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, NoTorch())
""",
    "blocked": "import sys\nsys.modules['torch'] = None\n"}


@pytest.mark.parametrize("how", list(NO_TORCH))
def test_star_import_without_torch(how):
    """The package and all of its names that need no torch come without it."""
    code = NO_TORCH[how] + """
from sparse_dense_matrix_gb300 import *
assert spmm_default_t_split(100, 1000, 50) >= 0 and "ExpertRoutes" not in globals()
"""
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert got.returncode == 0, got.stderr


def test_star_import_with_torch():
    code = "from sparse_dense_matrix_gb300 import *\nassert ExpertRoutes and dynamic_sync and spmm\n"
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert got.returncode == 0, got.stderr


def test_limits_and_refusals_of_the_later_calls():
    import ctypes

    import sparse_dense_matrix_gb300.dynamic as m
    ptr, L = ctypes.c_void_p(4096), m.lib        # never dereferenced: the checks come first
    rows = m._Rows(4096, 8192, 256, 64)

    def shape(B=1, Tq=4, Tk=64, Hq=4, Hk=2):
        return m._Shape(B, Tq, Tk, Hq, Hk, 64, 16, 2, 1, 1, 0.125, None)

    for limit in (0, -5, 10 ** 7 + 1):
        assert L.spmm_dynamic_check_wait_timeout(limit, None) == 1
    assert L.spmm_blocks_select_kept(shape(), rows, ptr, None, None, None, 0, None) == 1
    assert L.spmm_blocks_select_kept(shape(), rows, None, ptr, ptr, None, 0, None) == 1
    # more keys or rows than the limits: the means as the gradient
    for s in (shape(B=1 << 12, Tk=1 << 26, Hq=8, Hk=8), shape(B=1 << 20, Tq=1 << 10)):
        assert L.spmm_blocks_means(s, rows, -1, ptr, None) == 5
        assert L.spmm_blocks_backward(s, rows, rows, rows, ptr, ptr, ptr, rows, ptr, ptr, ptr, ptr,
                                      1 << 62, None) == 5
        assert L.spmm_blocks_backward_workspace(s) == 0
    # what the forward takes, the gradient takes: scratch for more pairs than 65535
    assert L.spmm_blocks_backward_workspace(shape(B=70000)) > 0
