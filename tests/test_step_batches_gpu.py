"""Single steps of the greatest batch that the calls take, 65535 sequences, each on its own slot in another order: every
sequence's result and state, against the formulas in float64.  fp32 sums of a few terms of unit size: 1e-5."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu
N = 65535


def inputs(dim):
    gen = torch.Generator(device="cuda").manual_seed(dim)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    slots = torch.randperm(N + 5, generator=gen, device="cuda")[:N].to(torch.int32)
    slots[[0, 4000, N - 1]] = torch.tensor([-1, N + 5, -7], dtype=torch.int32, device="cuda")
    return rn, slots, (slots >= 0) & (slots < N + 5)


def rest(slots, held):
    free = torch.ones(N + 5, dtype=torch.bool, device="cuda")
    free[slots[held].long()] = False
    return free


@pytest.mark.parametrize("dim", [4, 3])
def test_recurrence(dim):
    rn, slots, held = inputs(dim)
    x, r, i, lam, state = rn(N, 1, dim), rn(N, 1, dim), rn(N, 1, dim), rn(dim) - 3, rn(N + 5, dim)
    before = state.clone()
    y = binding.glr_step(x, r, i, lam, state, slots)
    g = -8 * torch.nn.functional.softplus(lam.double()) * torch.sigmoid(r[:, 0].double())
    at = slots[held].long()
    h = torch.exp(g)[held] * before[at].double() + (torch.sqrt(-torch.expm1(2 * g)) * torch.sigmoid(i[:, 0].double())
                                                    * x[:, 0].double())[held]
    assert float((y[held][:, 0] - h).abs().max()) <= 1e-5 and float((state[at] - h).abs().max()) <= 1e-5
    assert (y[~held] == 0).all() and torch.equal(state[rest(slots, held)], before[rest(slots, held)])


@pytest.mark.parametrize("dim", [4, 3])
def test_convolution(dim):
    rn, slots, held = inputs(dim + 8)
    x, w, b, state = rn(N, 1, dim), 0.5 * rn(dim, 4), rn(dim), rn(N + 5, 3, dim)
    before = state.clone()
    y = binding.conv_step(x, w, b, state, slots)
    at = slots[held].long()
    row = torch.cat([before[at], x[held]], 1)
    z = b.double() + (w.double().T * row.double()).sum(1)
    assert float((y[held][:, 0] - z * torch.sigmoid(z)).abs().max()) <= 1e-5
    assert torch.equal(state[at], row[:, 1:])
    assert (y[~held] == 0).all() and torch.equal(state[rest(slots, held)], before[rest(slots, held)])
