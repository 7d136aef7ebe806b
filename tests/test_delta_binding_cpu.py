"""What the delta rule's and the norm's Python calls do on the host, with stand-ins for tensors, devices and the library's
calls: no GPU is needed."""
import contextlib

import pytest
import torch

from selective_state_space_ssd_gb300 import binding


class Far:
    """A tensor on a device of the given index, as far as the checks of a call look at it."""

    def __init__(self, index):
        self.index, self.device = index, torch.device("cuda", index)

    def get_device(self):
        return self.index


@pytest.fixture
def current(monkeypatch):
    """The index of the current device, as a list of one that a test may change."""
    at = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    return at


def test_tensors_on_another_device_than_the_current_one_are_refused(current):
    a, b = Far(1), Far(1)
    with pytest.raises(ValueError, match="current"):
        binding._device(a, b, None)
    current[0] = 1
    assert binding._device(a, b, None) == 1
    with pytest.raises(ValueError, match="one CUDA device"):
        binding._device(a, Far(0))


def far_from(stream_index, current, monkeypatch):
    """Calls with stream= run as if on a stream of device `stream_index`; no tensor may be made, no kernel launched."""
    @contextlib.contextmanager
    def on(stream, device, *rest):
        before, current[0] = current[0], stream_index
        yield
        current[0] = before

    monkeypatch.setattr(binding, "_on", on)
    for name in ("ssd_delta_forward", "ssd_delta_backward", "ssd_delta_step", "ssd_norm_forward", "ssd_norm_backward"):
        monkeypatch.setattr(binding, name, lambda *a: pytest.fail("launched"))
    real = torch.Tensor.get_device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if real(t) < 0 else real(t))


@pytest.mark.parametrize("stream", [None, 0])
def test_calls_off_the_current_device_launch_nothing(stream, current, monkeypatch):
    far_from(0, current, monkeypatch)
    cfg = dict(dtype="bf16", gate_dtype="f32", batch=1, seqlen=3, nheads=1, value_heads=1, key_dim=8, value_dim=8)
    x = [torch.zeros((1, 3, 1, 8), dtype=torch.bfloat16) for _ in range(3)] + [torch.zeros((1, 3, 1)) for _ in range(2)]
    rows, stat, state = torch.zeros((4, 8)), torch.zeros(4), torch.zeros((1, 1, 8, 8))
    for call in (lambda: binding.delta_forward(cfg, *x, stream=stream),
                 lambda: binding.delta_backward(cfg, x[2], *x, stream=stream),
                 lambda: binding.delta_step(cfg, *x, state, stream=stream),
                 lambda: binding.norm_forward(rows, stream=stream),
                 lambda: binding.norm_backward(rows, rows, stat, stat, stream=stream)):
        with pytest.raises(ValueError, match="current"):
            call()
