"""GPU parity of the gated feed-forward (through the C ABI) with the formulas in float64.

Bounds, set before the first run.  h: fp32 sums over D (below 1e-5 of the sum's size at these sizes) rounded once to bf16,
half a step of 2^-7 of the value: max|gpu - ref| / max|ref| <= 4e-3.  The gradients are sums over terms with a factor dG or
dU that has been rounded to bf16 (2^-8 of each at most; the stash's 24 bits add 2^-15 to each of two factors) and are rounded
once more: 2^-7 of the sum's size where all roundings agree, as they can where the sum has one term: 8e-3."""
import numpy as np
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu


def make(m, d, f, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    c = dict(x=rn(m, d), wg=1.5 * rn(f, d) * d ** -0.5, wu=rn(f, d) * d ** -0.5, dh=rn(m, f))
    return {k: t.to(torch.bfloat16) for k, t in c.items()}


def act_of(g, act):
    if act == "silu":
        s = 1 / (1 + np.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    root = np.sqrt(2 / np.pi)
    t = np.tanh(root * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * root * (1 + 3 * 0.044715 * g * g)


def reference(c, act):
    f = {k: t.double().numpy() for k, t in c.items()}
    g, u = f["x"] @ f["wg"].T, f["x"] @ f["wu"].T
    a, s = act_of(g, act)
    dg, du = f["dh"] * u * s, f["dh"] * a
    return dict(h=a * u, dx=dg @ f["wg"] + du @ f["wu"], dwg=dg.T @ f["x"], dwu=du.T @ f["x"])


def check(name, got, ref, tol):
    x = got.double().cpu().numpy()
    assert x.shape == ref.shape and np.isfinite(x).all(), name
    err = float(np.abs(x - ref).max()) / max(float(np.abs(ref).max()), 1e-30)
    assert err <= tol, (name, err)


def compare(c, act, stash=True):
    ref = reference(c, act)
    d = {k: t.cuda() for k, t in c.items()}
    status = binding.delta_status()
    kept = binding.ffn_stash(d["x"], d["wg"]) if stash else None
    h = binding.ffn_forward(d["x"], d["wg"], d["wu"], act, stash=kept, status=status)
    g = binding.ffn_backward(d["dh"], d["x"], d["wg"], d["wu"], act, stash=kept, status=status)
    binding.check_status(status)
    check("h", h, ref["h"], 4e-3)
    for k in ("dx", "dwg", "dwu"):
        check(k, g[k], ref[k], 8e-3)
    return [h, *g.values()]


# one row; both sides of a tile of rows, of columns and of a step of the sum; more tiles than SMs
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,d,f", [(1, 8, 8), (1, 64, 128), (2, 256, 136), (7, 72, 120), (16, 128, 256), (17, 264, 64),
                                   (63, 8, 512), (64, 320, 192), (65, 56, 8), (127, 248, 384), (128, 64, 128),
                                   (129, 192, 264), (200, 512, 1032), (257, 136, 72), (300, 1032, 520), (1000, 520, 776)])
def test_matches_float64(m, d, f, act):
    compare(make(m, d, f, 1), act)


@pytest.mark.parametrize("m,d,f", [(2100, 328, 2568), (1100, 1544, 2568), (1100, 72, 2568)])
def test_more_tiles_than_blocks(m, d, f):
    """An odd number of row tiles, whose last has no neighbour; wide and narrow tiles, forward and backward."""
    compare(make(m, d, f, 2), "silu")


@pytest.mark.parametrize("m,d,f", [(1, 8, 1024), (65, 264, 2056), (130, 40, 5000), (300, 72, 4104), (257, 520, 1032)])
def test_long_sums_of_few_rows(m, d, f):
    """dx of sums that are taken in pieces."""
    compare(make(m, d, f, 9), "gelu")


@pytest.mark.parametrize("m,d,f", [(150, 264, 392), (70, 136, 2568)])
def test_stash_changes_no_bit(m, d, f):
    c = make(m, d, f, 3)
    a, b = compare(c, "silu"), compare(c, "silu", stash=False)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_behind_the_last_are_left_alone():
    c = make(130, 128, 200, 4)
    d = {k: t.cuda() for k, t in c.items()}
    prob = binding.ffn_problem(d["x"], d["wg"])
    h = torch.full((140, 200), 7.0, device="cuda", dtype=torch.bfloat16)
    n = binding.ssd_ffn_workspace_size(prob, False)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    binding.ssd_ffn_forward(prob, d["x"], d["wg"], d["wu"], h, None, 0, ws, n)
    assert (h[130:] == 7).all()
    assert torch.equal(h[:130], binding.ffn_forward(d["x"], d["wg"], d["wu"]))
    assert binding.ssd_read_status(ws) == (0, 0)


def test_strided_rows_and_leading_dimensions():
    c = make(60, 64, 96, 5)
    d = {k: t.cuda() for k, t in c.items()}
    want = compare(c, "silu")
    room = torch.full((60, 200), float("nan"), device="cuda", dtype=torch.bfloat16)
    room[:, 136:] = d["x"]
    x = room[:, 136:]
    stash = binding.ffn_stash(x, d["wg"])
    h = binding.ffn_forward(x, d["wg"], d["wu"], stash=stash)
    g = binding.ffn_backward(d["dh"], x, d["wg"], d["wu"], stash=stash)
    assert torch.equal(h, want[0]) and all(torch.equal(a, b) for a, b in zip(g.values(), want[1:]))
    assert torch.equal(binding.ffn_forward(d["x"].view(3, 20, 64), d["wg"], d["wu"]).view(60, 96), h)


def test_a_nan_stays_in_its_row():
    c = make(70, 64, 96, 6)
    ref = reference(c, "silu")
    c["x"][33, 5] = float("nan")
    d = {k: t.cuda() for k, t in c.items()}
    h = binding.ffn_forward(d["x"], d["wg"], d["wu"])
    dx = binding.ffn_backward(d["dh"], d["x"], d["wg"], d["wu"])["dx"]
    rest = [r for r in range(70) if r != 33]
    assert h[33].isnan().all()
    check("h", h[rest], ref["h"][rest], 4e-3)
    check("dx", dx[rest], ref["dx"][rest], 8e-3)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_far_from_zero(act):
    c = make(32, 8, 16, 7)
    c["wg"] = (c["wg"].float() * 60).to(torch.bfloat16)
    compare(c, act)


def test_gradients_against_differences():
    c = make(3, 8, 8, 8)
    f = {k: t.double().numpy() for k, t in c.items()}

    def loss(**over):
        v = {**f, **over}
        return float((act_of(v["x"] @ v["wg"].T, "gelu")[0] * (v["x"] @ v["wu"].T) * f["dh"]).sum())

    d = {k: t.cuda() for k, t in c.items()}
    g = binding.ffn_backward(d["dh"], d["x"], d["wg"], d["wu"], "gelu")
    for leaf, name in (("x", "dx"), ("wg", "dwg"), ("wu", "dwu")):
        num = np.zeros_like(f[leaf])
        for at in np.ndindex(num.shape):
            step = np.zeros_like(num)
            step[at] = 1e-5
            num[at] = (loss(**{leaf: f[leaf] + step}) - loss(**{leaf: f[leaf] - step})) / 2e-5
        check(name, g[name], num, 8e-3)


def test_same_bits_again_on_another_stream_and_in_a_graph():
    c = make(300, 136, 264, 9)
    d = {k: t.cuda() for k, t in c.items()}

    def both():
        stash = binding.ffn_stash(d["x"], d["wg"])
        h = binding.ffn_forward(d["x"], d["wg"], d["wu"], stash=stash)
        return [h, *binding.ffn_backward(d["dh"], d["x"], d["wg"], d["wu"], stash=stash).values()]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = binding.ffn_forward(d["x"], d["wg"], d["wu"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_two_to_the_31():
    m, d, f = (1 << 31) // 4096 + 300, 64, 4096
    gen = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn((m, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    wg, wu = (torch.randn((f, d), generator=gen, device="cuda", dtype=torch.bfloat16) * 0.1 for _ in range(2))
    dh = torch.randn((m, f), generator=gen, device="cuda", dtype=torch.bfloat16)
    stash = binding.ffn_stash(x, wg)
    h = binding.ffn_forward(x, wg, wu, stash=stash)
    dx = binding.ffn_backward(dh, x, wg, wu, stash=stash)["dx"]
    for a, b in ((0, 256), (m - 300, m)):
        part = {"x": x[a:b].cpu(), "wg": wg.cpu(), "wu": wu.cpu(), "dh": dh[a:b].cpu()}
        ref = reference(part, "silu")
        check("h", h[a:b], ref["h"], 4e-3)
        check("dx", dx[a:b], ref["dx"], 8e-3)
