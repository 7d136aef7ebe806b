"""The convolution's autograd function where the taps before a piece carry gradients: taps with and without a batch axis,
pieces of fewer steps than taps.  On the CPU with the library's calls replaced by the formulas in float64, on the GPU with
the calls themselves in fp32: sums of at most 10 terms (two sequences of five steps) of up to 20 in size, whose factors pass
an exponential and a reciprocal that are good to 2^-22 each: 10 x 20 x 5e-7 = 1e-4."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding
from selective_state_space_ssd_gb300.recurrent_block import ShortConv


def plain(x, weight, bias, taps):
    """y and the taps that follow, of x [T, D] or [b, T, D]; the taps that follow are [b, K - 1, D]."""
    k, steps = weight.shape[1], x.shape[-2]
    row = torch.cat([taps.reshape(-1, k - 1, x.shape[-1]), x.reshape(-1, steps, x.shape[-1])], 1)
    z = bias + sum(weight[:, j] * row[:, j:j + steps] for j in range(k))
    return (z * torch.sigmoid(z)).reshape(x.shape), row[:, steps:]


def conv_forward(x, weight, bias, activation, taps):
    with torch.no_grad():
        return plain(x, weight, bias, taps)


def conv_backward(dy, x, weight, bias, activation, taps):
    with torch.enable_grad():
        leaves = [t.detach().clone().requires_grad_() for t in (x, weight, bias, taps)]
        grads = torch.autograd.grad(plain(*leaves)[0], leaves, dy)
    return dict(zip(("dx", "dw", "db", "dtaps"), grads))


CASES = [(k, steps, x_axis, taps_axis) for k in (2, 3, 4) for steps in (1, 2, 3, 5) for x_axis in (0, 1, 2) for taps_axis in (0, 1)
         if x_axis < 2 or taps_axis]


def compare(k, steps, x_axis, taps_axis, dtype, device, tol):
    """x_axis: 0: [T, D], else a batch of so many; taps_axis: 0: [K - 1, D]."""
    gen = torch.Generator().manual_seed(k * 10 + steps)
    rn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64).to(dtype).to(device)  # noqa: E731
    b, dim = max(x_axis, 1), 12
    values = (rn(*((b,) if x_axis else ()), steps, dim), rn(dim, k), rn(dim), rn(*((b,) if taps_axis else ()), k - 1, dim))
    dy, dlast = rn(*values[0].shape), rn(b, k - 1, dim)
    got, want = [t.clone().requires_grad_() for t in values], [t.double().clone().requires_grad_() for t in values]
    y, last = ShortConv.apply(*got)
    yw, lastw = plain(*want)
    assert last.shape == lastw.shape
    grads = torch.autograd.grad((y * dy).sum() + (last * dlast).sum(), got)
    wants = torch.autograd.grad((yw * dy.double()).sum() + (lastw * dlast.double()).sum(), want)
    for a, w in zip((y, last, *grads), (yw, lastw, *wants)):
        assert a.shape == w.shape and float((a.detach().double() - w.detach()).abs().max()) <= tol


@pytest.mark.parametrize("k,steps,x_axis,taps_axis", CASES)
def test_taps_gradients(monkeypatch, k, steps, x_axis, taps_axis):
    monkeypatch.setattr(binding, "conv_forward", conv_forward)
    monkeypatch.setattr(binding, "conv_backward", conv_backward)
    compare(k, steps, x_axis, taps_axis, torch.float64, "cpu", 1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("k,steps,x_axis,taps_axis", CASES)
def test_taps_gradients_of_the_calls(k, steps, x_axis, taps_axis):
    compare(k, steps, x_axis, taps_axis, torch.float32, "cuda", 1e-4)
