"""The binding's host side without a GPU: devices of streams."""
import types


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
