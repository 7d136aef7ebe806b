"""The mixer block's autograd functions, with the library's calls replaced by the same formulas on the CPU whose results,
like the library's, carry no history: no GPU is needed."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding
from selective_state_space_ssd_gb300.delta_mixer import DeltaRule, LayerNorm


def norm_forward(x, weight, bias, eps):
    with torch.no_grad():
        mean = x.mean(-1)
        rstd = (x.var(-1, unbiased=False) + eps).rsqrt()
        return (x - mean[:, None]) * rstd[:, None] * weight + bias, mean, rstd


def norm_backward(dy, x, mean, rstd, weight):
    with torch.no_grad():
        h, g = (x - mean[:, None]) * rstd[:, None], dy * weight
        dx = rstd[:, None] * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
        return dict(dx=dx, dw=(dy * h).sum(0), db=dy.sum(0))


@pytest.fixture
def calls(monkeypatch):
    """One step of one head whose o is v * beta, and a norm."""
    monkeypatch.setattr(binding, "norm_forward", norm_forward)
    monkeypatch.setattr(binding, "norm_backward", norm_backward)
    monkeypatch.setattr(binding, "delta_stash", lambda *a, **k: torch.zeros(1))
    monkeypatch.setattr(binding, "delta_forward", lambda cfg, q, k, v, g, beta, **o: ((v * beta[..., None]).detach(), None))
    monkeypatch.setattr(binding, "delta_backward", lambda cfg, do, q, k, v, g, beta, **o: dict(
        dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=(do * beta[..., None]).detach(), dg=torch.zeros_like(g),
        dbeta=(do * v).sum(-1).detach()))


def losses(kind):
    gen = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    if kind == "norm":
        x, w = rn(3, 5).requires_grad_(), rn(5).requires_grad_()
        y, leaves = LayerNorm.apply(x, w, rn(5).requires_grad_(), 1e-5), (x, w)
    else:
        x, beta = rn(1, 1, 1, 4).requires_grad_(), rn(1, 1, 1).requires_grad_()
        y, leaves = DeltaRule.apply({}, rn(1, 1, 1, 4), rn(1, 1, 1, 4), x, rn(1, 1, 1), beta), (x, beta)
    return y, leaves, rn(*y.shape)


@pytest.mark.parametrize("linear", [True, False])
@pytest.mark.parametrize("kind", ["norm", "delta"])
@pytest.mark.parametrize("leaf", [0, 1])
def test_second_derivatives_are_refused(calls, kind, leaf, linear):
    """A penalty on a gradient: the loss's own gradient may be a constant (linear) or depend on the output."""
    y, leaves, c = losses(kind)
    first = torch.autograd.grad((y * c).sum() if linear else y.square().sum(), leaves[leaf], create_graph=True)[0]
    penalty = first.square().sum() + sum(t.sum() for t in leaves)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(penalty, leaves)
    y, leaves, c = losses(kind)
    first = torch.autograd.grad((y * c).sum() if linear else y.square().sum(), leaves[leaf], create_graph=True)[0]
    with pytest.raises(RuntimeError, match="second derivative"):
        (first.square().sum() + sum(t.sum() for t in leaves)).backward()


@pytest.mark.parametrize("kind", ["norm", "delta"])
def test_first_derivatives_are_the_same_with_and_without_a_graph(calls, kind):
    y, leaves, c = losses(kind)
    loss = (y * c).sum()
    graph = torch.autograd.grad(loss, leaves, create_graph=True)
    plain = torch.autograd.grad(loss, leaves)
    for a, b in zip(graph, plain):
        assert torch.equal(a, b) and not b.requires_grad
    if kind == "norm":
        x, w = (t.detach().requires_grad_() for t in leaves)
        want = torch.autograd.grad((torch.nn.functional.layer_norm(x, (5,), w, None, 1e-5) * c).sum(), (x, w))
        for a, b in zip(plain, want):
            assert torch.allclose(a, b, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_norm_without_a_weight_or_a_bias(calls, monkeypatch, weight, bias):
    one, zero = torch.ones(5, dtype=torch.float64), torch.zeros(5, dtype=torch.float64)
    monkeypatch.setattr(binding, "norm_forward", lambda x, w, b, eps: norm_forward(x, one if w is None else w,
                                                                                  zero if b is None else b, eps))
    monkeypatch.setattr(binding, "norm_backward", lambda dy, x, m, r, w: norm_backward(dy, x, m, r, one if w is None else w))
    gen = torch.Generator().manual_seed(2)
    x, w, b, c = (torch.randn(s, generator=gen, dtype=torch.float64).requires_grad_() for s in ((3, 5), (5,), (5,), (3, 5)))
    w, b = w if weight else None, b if bias else None
    leaves = [t for t in (x, w, b) if t is not None]
    got = torch.autograd.grad((LayerNorm.apply(x, w, b, 1e-5) * c).sum(), leaves)
    want = torch.autograd.grad((torch.nn.functional.layer_norm(x, (5,), w, b, 1e-5) * c).sum(), leaves)
    for g, r in zip(got, want):
        assert torch.allclose(g, r, rtol=1e-10, atol=1e-12)
