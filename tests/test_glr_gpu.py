"""GPU parity of the gated linear recurrence (through the C ABI) with the formulas in float64, step by step.

Bounds (max|gpu - ref| / max|ref|), set before the first run.  fp32 outputs: a gate's exponentials and the state's rounding
leave up to 2^-23 a step, which a state carries on for 1 / (1 - a) steps; decays of up to 0.999 make that 1000 x 6e-8 = 6e-5
at worst where all errors point one way, and 1e-6 where they do not: 2e-5.  dlam sums over all steps: 5e-5.  bf16 outputs are
rounded once more: half a step of 2^-8 of the value, 4e-3."""
import numpy as np
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {torch.float32: 2e-5, torch.bfloat16: 4e-3}


def make(lead, dim, io, seed, n):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    a = 0.9 + 0.099 * torch.rand(dim, generator=gen)
    c = dict(x=rn(*lead, dim), r=1.5 * rn(*lead, dim), i=1.5 * rn(*lead, dim), dy=rn(*lead, dim))
    c = {k: t.to(TYPES[io]) for k, t in c.items()}
    return dict(c, lam=torch.log(torch.expm1(-torch.log(a) / 8)), h0=rn(n, dim), dh=rn(n, dim))


def sig(z):
    return 1 / (1 + np.exp(-z))


def walk(x, r, i, lam, h0, dy=None, dh=None, scale=8.0):
    """One sequence [T, D] in float64: y, the last state and (with dy) the gradients of <dy, y> + <dh, last>."""
    rs, gi = sig(r), sig(i)
    g = -scale * np.log1p(np.exp(lam)) * rs
    a, m = np.exp(g), np.sqrt(-np.expm1(2 * g))
    h, ys = h0.copy(), np.zeros_like(x)
    for t in range(x.shape[0]):
        h = a[t] * h + m[t] * gi[t] * x[t]
        ys[t] = h
    if dy is None:
        return dict(y=ys, last=h)
    d, out = dh.copy(), {k: np.zeros_like(x) for k in ("dx", "dr", "di")}
    dlam = np.zeros_like(lam)
    for t in reversed(range(x.shape[0])):
        d = d + dy[t]
        before = ys[t - 1] if t else h0
        dg = d * (a[t] * before - a[t] ** 2 / m[t] * gi[t] * x[t])
        out["dx"][t] = d * m[t] * gi[t]
        out["di"][t] = d * m[t] * x[t] * gi[t] * (1 - gi[t])
        out["dr"][t] = dg * g[t] * (1 - rs[t])
        dlam += dg * -scale * sig(lam) * rs[t]
        d = a[t] * d
    return dict(y=ys, last=h, dlam=dlam, dh0=d, **out)


def reference(c, bounds=None, h0=True, dh=True):
    f = {k: t.double().numpy() for k, t in c.items()}
    zero = np.zeros_like(f["h0"][0])
    x = {k: f[k].reshape(-1, f[k].shape[-1]) for k in ("x", "r", "i", "dy")}
    if bounds is None:
        steps = c["x"].shape[-2]
        bounds = [steps * n for n in range(f["h0"].shape[0] + 1)]
    ref = {k: np.zeros_like(x["x"]) for k in ("y", "dx", "dr", "di")}
    ref.update(last=np.zeros_like(f["h0"]), dh0=np.zeros_like(f["h0"]), dlam=np.zeros_like(f["lam"]))
    for n, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        w = walk(*(x[k][a:b] for k in ("x", "r", "i")), f["lam"], f["h0"][n] if h0 else zero, x["dy"][a:b],
                 f["dh"][n] if dh else zero)
        for k in ("y", "dx", "dr", "di"):
            ref[k][a:b] = w[k]
        ref["last"][n], ref["dh0"][n] = w["last"], w["dh0"]
        ref["dlam"] += w["dlam"]
    for k in ("y", "dx", "dr", "di"):
        ref[k] = ref[k].reshape(f["x"].shape)
    return ref


def check(name, got, ref, tol=None):
    x = got.double().cpu().numpy()
    assert x.shape == ref.shape and np.isfinite(x).all(), name
    err = float(np.abs(x - ref).max()) / max(float(np.abs(ref).max()), 1e-30)
    assert err <= (tol or TOL[got.dtype]), (name, err)


def compare(c, cu=None, bounds=None, h0=True, dh=True, stash=True):
    ref = reference(c, bounds, h0, dh)
    d = {k: t.cuda() for k, t in c.items()}
    first, seed = d["h0"] if h0 else None, d["dh"] if dh else None
    kept = binding.glr_stash(d["x"]) if stash else None
    y, last = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], first, cu_seqlens=cu, stash=kept)
    g = binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], seed, first, cu_seqlens=cu, stash=kept)
    torch.cuda.synchronize()
    check("y", y, ref["y"])
    check("h_final", last, ref["last"])
    for k in ("dx", "dr", "di"):
        check(k, g[k], ref[k])
    check("dlam", g["dlam"], ref["dlam"], 5e-5)
    if h0:
        check("dh0", g["dh0"], ref["dh0"])
    else:
        assert g["dh0"] is None
    return y, last, g


# one step, both sides of a run, a mark, a tile and several tiles; widths on both sides of a slab, whole and ragged pieces
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,steps,dim", [(1, 1, 1), (2, 2, 3), (1, 7, 64), (3, 8, 65), (2, 9, 32), (1, 31, 33), (2, 32, 8),
                                         (1, 33, 72), (2, 63, 130), (1, 64, 128), (2, 65, 40), (1, 97, 63), (2, 129, 96), (300, 5, 16), (50, 33, 40),
                                         (1, 257, 16), (5, 300, 100), (1, 1000, 24), (2, 517, 200)])
def test_matches_float64(n, steps, dim, io):
    compare(make((n, steps), dim, io, 1, n))


@pytest.mark.parametrize("h0,dh,stash", [(False, False, True), (True, False, False), (False, True, False)])
def test_without_first_state_final_gradient_or_stash(h0, dh, stash):
    c = make((2, 150), 96, "bf16", 2, 2)
    compare(c, h0=h0, dh=dh, stash=stash)


def test_stash_changes_no_bit():
    c = make((2, 131), 72, "bf16", 3, 2)
    a, b = compare(c), compare(c, stash=False)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,dim", [([5], 8), ([1, 1, 1], 64), ([0, 33, 0, 64, 1, 0], 70), ([100, 7, 193], 96),
                                         ([64, 64, 64], 40), ([3] * 50, 33), ([0, 0, 9], 16), ([500, 0, 2, 31], 129)])
def test_packed_matches_float64(lengths, dim, io):
    bounds = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    c = make((bounds[-1],), dim, io, 4, len(lengths))
    compare(c, torch.tensor(bounds, dtype=torch.int32, device="cuda"), bounds)
    compare(c, torch.tensor(bounds, dtype=torch.int32, device="cuda"), bounds, h0=False, dh=False, stash=False)


def test_steps_of_no_sequence_are_zero_and_touch_nothing():
    bounds = [13, 20, 90]
    c = make((120,), 72, "bf16", 5, 2)
    for k in ("x", "r", "i", "dy"):
        c[k][:13] = float("nan")
        c[k][90:] = float("inf")
    clean = {k: t.clone() for k, t in c.items()}
    for k in ("x", "r", "i", "dy"):
        clean[k][:13] = clean[k][90:] = 0
    ref = reference(clean, bounds)
    d = {k: t.cuda() for k, t in c.items()}
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y, last = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"], cu_seqlens=cu)
    g = binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], d["dh"], d["h0"], cu_seqlens=cu)
    check("y", y, ref["y"])
    check("last", last, ref["last"])
    for k in ("dx", "dr", "di", "dh0"):
        check(k, g[k], ref[k])
    check("dlam", g["dlam"], ref["dlam"], 5e-5)
    for t in (y, g["dx"], g["dr"], g["di"]):
        assert not t[:13].any() and not t[90:].any()


def test_a_nan_stays_in_its_sequence_and_channel():
    bounds = [0, 40, 100, 170]
    c = make((170,), 64, "f32", 6, 3)
    ref = reference(c, bounds)
    c["x"][55, 7] = float("nan")
    c["r"][60, 9] = float("nan")
    d = {k: t.cuda() for k, t in c.items()}
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y, last = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"], cu_seqlens=cu)
    g = binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], d["dh"], d["h0"], cu_seqlens=cu)
    y, last = y.cpu(), last.cpu()
    assert y[55:100, 7].isnan().all() and y[60:100, 9].isnan().all() and last[1, 7].isnan()
    hit = torch.zeros(170, 64, dtype=torch.bool)
    hit[40:100, [7, 9]] = True
    for name, t in (("y", y), ("dx", g["dx"].cpu()), ("dr", g["dr"].cpu()), ("di", g["di"].cpu())):
        rest = torch.where(hit, torch.zeros(()), t)
        check(name, rest, np.where(hit.numpy(), 0, ref[name]))


def test_bounds_that_leave_the_axis_are_clamped():
    c = make((50,), 24, "f32", 7, 2)
    d = {k: t.cuda() for k, t in c.items()}
    run = lambda b: binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"],  # noqa: E731
                                        cu_seqlens=torch.tensor(b, dtype=torch.int32, device="cuda"))
    got, want = run([-5, 20, 1000]), run([0, 20, 50])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gates_far_from_zero_are_finite():
    c = make((1, 40), 32, "f32", 8, 1)
    for k, v in (("r", 200.0), ("i", 200.0)):
        c[k][0, :10] = v
        c[k][0, 10:20] = -v
    c["lam"][:4] = torch.tensor([-200.0, -30.0, 30.0, 80.0])
    c["r"][0, 25] = -torch.inf
    c["i"][0, 26] = -torch.inf
    c["r"][0, 27] = torch.inf
    d = {k: t.cuda() for k, t in c.items()}
    y, last = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"])
    g = binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], d["dh"], d["h0"])
    with np.errstate(all="ignore"):
        ref = reference(c)
    check("y", y, ref["y"])
    check("last", last, ref["last"])
    for k in ("dx", "di", "dh0"):
        check(k, g[k], ref[k])
    assert all(t.isfinite().all() for t in g.values())
    ok = np.isfinite(ref["dr"])  # (where 1 - a^2 rounds to nothing the float64 formula divides by zero)
    assert ok.mean() > 0.5
    check("dr", torch.where(torch.from_numpy(ok), g["dr"].cpu(), 0.0), np.where(ok, ref["dr"], 0))


@pytest.mark.parametrize("io,dim,wide", [("bf16", 64, 192), ("bf16", 40, 83), ("bf16", 33, 70), ("f32", 33, 70), ("f32", 64, 128)])
def test_strided_inputs(io, dim, wide):
    c = make((3, 70), dim, io, 9, 3)
    d = {k: t.cuda() for k, t in c.items()}
    want = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"])
    back = binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], d["dh"], d["h0"])
    for k in ("x", "r", "i"):
        room = torch.full((3, 70, wide), float("nan"), dtype=d[k].dtype, device="cuda")
        room[..., wide - dim:] = d[k]
        d[k] = room[..., wide - dim:]
    got = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    again = binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], d["dh"], d["h0"])
    assert all(torch.equal(back[k], again[k]) for k in back)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,steps,dim", [(1, 1, 64), (3, 1, 33), (5, 7, 100), (2, 3, 4096)])
def test_steps_match_the_scan(n, steps, dim, io):
    c = make((n, steps), dim, io, 10, n)
    ref = reference(c)
    d = {k: t.cuda() for k, t in c.items()}
    slots = torch.tensor([2 * j + 1 for j in range(n)], dtype=torch.int32, device="cuda")
    state = torch.full((2 * n + 1, dim), 7.0, device="cuda")
    state[slots.long()] = d["h0"]
    y = binding.glr_step(d["x"], d["r"], d["i"], d["lam"], state, slots)
    check("y", y, ref["y"])
    check("state", state[slots.long()], ref["last"])
    assert (state[::2] == 7).all()
    own = d["h0"].clone()  # without slot numbers: sequence n has slot n
    assert torch.equal(binding.glr_step(d["x"], d["r"], d["i"], d["lam"], own), y)
    assert torch.equal(own, state[slots.long()])


def test_places_without_a_sequence():
    c = make((4, 2), 48, "bf16", 11, 4)
    d = {k: t.cuda() for k, t in c.items()}
    state = d["h0"].clone()
    y = binding.glr_step(d["x"], d["r"], d["i"], d["lam"], state, torch.tensor([1, -1, 9, 0], dtype=torch.int32, device="cuda"))
    assert not y[1:3].any() and y[0].any() and y[3].any()
    assert torch.equal(state[2:], d["h0"][2:]) and not torch.equal(state[:2], d["h0"][:2])


def test_gradients_against_differences():
    c = make((1, 12), 6, "f32", 12, 1)
    f = {k: t.double().numpy() for k, t in c.items()}

    def loss(**over):
        v = {**f, **over}
        w = walk(v["x"][0], v["r"][0], v["i"][0], v["lam"], v["h0"][0])
        return float((w["y"] * f["dy"][0]).sum() + (w["last"] * f["dh"][0]).sum())

    d = {k: t.cuda() for k, t in c.items()}
    g = binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], d["dh"], d["h0"])
    for leaf, name in (("x", "dx"), ("r", "dr"), ("i", "di"), ("lam", "dlam"), ("h0", "dh0")):
        num = np.zeros_like(f[leaf])
        for at in np.ndindex(num.shape):
            step = np.zeros_like(num)
            step[at] = 1e-5
            num[at] = (loss(**{leaf: f[leaf] + step}) - loss(**{leaf: f[leaf] - step})) / 2e-5
        check(name, g[name], num, 5e-5)


def test_long_sequences_in_many_tiles():
    c = make((1, 5000), 64, "f32", 13, 1)
    compare(c)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,steps,dim", [(1, 3000, 70), (3, 1400, 33), (1, 1700, 2624)])
def test_more_tiles_than_blocks_that_share_them(n, steps, dim, io):
    """Few channels (blocks of many warps) and many of them (of few), over several rounds of a cluster."""
    compare(make((n, steps), dim, io, 14, n))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,dim", [([1200, 0, 1, 700, 65, 1100], 70), ([2900, 3], 64), ([129] * 20 + [0, 1], 33)])
def test_packed_over_several_rounds(lengths, dim, io):
    bounds = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    compare(make((bounds[-1],), dim, io, 15, len(lengths)), torch.tensor(bounds, dtype=torch.int32, device="cuda"), bounds)


def test_same_bits_again_on_another_stream_and_in_a_graph():
    c = make((2, 300), 128, "bf16", 14, 2)
    d = {k: t.cuda() for k, t in c.items()}

    def both():
        stash = binding.glr_stash(d["x"])
        y, last = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"], stash=stash)
        return [y, last, *binding.glr_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], d["dh"], d["h0"], stash=stash).values()]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, last = binding.glr_forward(d["x"], d["r"], d["i"], d["lam"], d["h0"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0]) and torch.equal(last, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_two_to_the_31():
    dim, steps = 4096, (1 << 31) // 4096 + 40
    gen = torch.Generator(device="cuda").manual_seed(15)
    x = torch.randn((steps, dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    lam = torch.full((dim,), -4.0, device="cuda")
    h0 = torch.zeros((2, dim), device="cuda")
    cu = torch.tensor([0, steps - 100, steps], dtype=torch.int32, device="cuda")
    y, last = binding.glr_forward(x, x, x, lam, h0, cu_seqlens=cu)
    g = binding.glr_backward(x, x, x, x, lam, cu_seqlens=cu)
    tail = x[steps - 100:].clone()
    y2, last2 = binding.glr_forward(tail, tail, tail, lam, h0[:1])
    g2 = binding.glr_backward(tail, tail, tail, tail, lam)
    # (runs of the short call begin at other steps, so its sums are joined in another order)
    check("y", y[steps - 100:], y2.double().cpu().numpy())
    check("last", last[1:], last2.double().cpu().numpy())
    for k in ("dx", "dr", "di"):
        check(k, g[k][steps - 100:], g2[k].double().cpu().numpy())
