"""The gated feed-forward where G is far from zero, up to what bf16 inputs hold, against float64.

Bounds, set before the first run.  x holds G itself in one column (the weight's is 1) and 1 in another, so that G and U are
exact.  h: the activation in fp32 (below 1e-4 of its value: z of e^z is rounded at 2^-24 of at most 88) rounded once to bf16,
2^-8: 4.1e-3 of the value.  Gradients: dG and dU rounded to bf16 and the result once more, 2^-7; G from the stash is off by
2^-15 of its value, so e^z by z' |g| 2^-15 <= 3 z 2^-15 of its value, 8e-3 at z = 88: 1.6e-2 of the sum of the terms' sizes.
Where e^z is beyond fp32's range the activation and its slope are 0 or 1 exactly; next to that, values below 1e-32 may have
been flushed."""
import numpy as np
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu

FAR = [0.3, 3.0, 8.0, 20.0, 60.0, 87.0, 100.0, 1e4, 1e10, 1e11, 1e12, 1e13, 1e19, 5e19, 1e25, 1e30, 1e36]


def act_of(g, act):
    """The activation and its slope, in float64, from e^-|z|, which never overflows."""
    if act == "silu":
        z, dz = g, np.ones_like(g)
    else:
        c, k = 2 * np.sqrt(2 / np.pi), 0.044715
        z, dz = c * (g + k * g ** 3), c * (1 + 3 * k * g * g)
    e = np.exp(-np.abs(z))
    q, rest = np.where(z > 0, 1, e) / (1 + e), np.where(z > 0, e, 1) / (1 + e)
    return g * q, q + np.where(q * rest > 0, g * dz, 0) * q * rest


def inputs(values, hidden, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    m, d = len(values), 16
    x, wg, wu = torch.zeros(m, d), torch.zeros(hidden, d), torch.zeros(hidden, d)
    x[:, 0], x[:, 1] = torch.tensor(values, dtype=torch.float64).float(), 1
    wg[:, 0], wu[:, 1] = 1, rn(hidden)
    return {k: t.to(torch.bfloat16) for k, t in dict(x=x, wg=wg, wu=wu, dh=rn(m, hidden)).items()}


def passes(c, act, stashed):
    d = {k: t.cuda() for k, t in c.items()}
    stash = binding.ffn_stash(d["x"], d["wg"]) if stashed else None
    h = binding.ffn_forward(d["x"], d["wg"], d["wu"], act, stash=stash)
    g = binding.ffn_backward(d["dh"], d["x"], d["wg"], d["wu"], act, stash=stash)
    return {k: t.double().cpu().numpy() for k, t in dict(g, h=h).items()}


def bounded(name, got, ref, size, tol, floor):
    big = np.abs(ref) > 3.4e38  # (bf16 ends at 3.39e38: a gradient beyond it is infinite)
    bad = np.where(big, got != np.sign(ref) * np.inf, ~(np.abs(np.where(big, 0, got) - np.where(big, 0, ref)) <= tol * size + floor))
    assert not bad.any(), (name, got[bad][:4], ref[bad][:4], size[bad][:4] if np.ndim(size) else size)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("value", FAR)
def test_one_row(value, sign, act):
    c = inputs([sign * value], 24, 1)
    f = {k: t.double().numpy() for k, t in c.items()}
    got = passes(c, act, stashed=True)
    g, u = f["x"][:, :1] * f["wg"].T[:1], f["wu"].T[1:2]
    a, s = act_of(g, act)
    dg, du = f["dh"] * u * s, f["dh"] * a
    floor = 1e-32 if value <= 100 else 0.0
    bounded("h", got["h"], a * u, np.abs(a * u), 4.1e-3, floor)
    bounded("dwg", got["dwg"], dg.T @ f["x"], np.abs(dg).T @ np.abs(f["x"]), 1.6e-2, 100 * floor)
    bounded("dwu", got["dwu"], du.T @ f["x"], np.abs(du).T @ np.abs(f["x"]), 1.6e-2, 100 * floor)
    bounded("dx", got["dx"], dg @ f["wg"] + du @ f["wu"], np.abs(dg) @ np.abs(f["wg"]) + np.abs(du) @ np.abs(f["wu"]),
            1.6e-2, 100 * floor)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("stashed", [True, False])
def test_rows_of_many_tiles(act, stashed):
    """Row by row, where the forward is walked over in tiles (more of them than SMs)."""
    values = [s * v for v in FAR[:-1] for s in (1, -1)]
    c = inputs([values[i % len(values)] for i in range(1100)], 2568, 2)
    f = {k: t.double().numpy() for k, t in c.items()}
    got = passes(c, act, stashed)
    g, u = f["x"][:, :1] * f["wg"].T[:1], f["wu"].T[1:2]
    a, s = act_of(g, act)
    dg, du = f["dh"] * u * s, f["dh"] * a
    bounded("h", got["h"], a * u, np.abs(a * u), 4.1e-3, 1e-32)
    bounded("dx", got["dx"], dg @ f["wg"] + du @ f["wu"], np.abs(dg) @ np.abs(f["wg"]) + np.abs(du) @ np.abs(f["wu"]),
            1.6e-2, 1e-28)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_a_nan_is_handed_on(act):
    c = inputs([float("nan"), 1.0], 16, 3)
    got = passes(c, act, stashed=True)
    assert np.isnan(got["h"][0]).all() and np.isnan(got["dx"][0, 0]) and np.isfinite(got["h"][1]).all()
    assert np.isfinite(got["dx"][1]).all() and np.isnan(got["dwg"][:, 0]).all()
