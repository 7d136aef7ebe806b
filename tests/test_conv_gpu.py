"""GPU parity of the causal short convolution (through the C ABI) with the formulas in float64.

Bounds (max|gpu - ref| / max|ref|), set before the first run: sums of up to five fp32 terms and an exponential leave about
1e-6, the sums over all steps for the weight less than 1e-5: 2e-5 for fp32 outputs.  bf16 outputs are rounded once: half a
step of 2^-8 of the value, 4e-3.  The taps are copies: equal."""
import numpy as np
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {torch.float32: 2e-5, torch.bfloat16: 4e-3}


def make(lead, dim, k, io, wt, seed, n):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    c = {name: t.to(TYPES[io]) for name, t in dict(x=rn(*lead, dim), dy=rn(*lead, dim), taps=rn(n, k - 1, dim)).items()}
    return dict(c, w=(rn(dim, k) * 0.7).to(TYPES[wt]), b=rn(dim).to(TYPES[wt]))


def one(x, w, b, taps, silu, dy):
    """One sequence [T, D] in float64, with its gradients."""
    k = w.shape[1]
    row = np.concatenate([taps, x])
    steps = x.shape[0]
    z = b + sum(w[:, j] * row[j:j + steps] for j in range(k))
    s = 0.5 * (1 + np.tanh(0.5 * z))
    y, dz = (z * s, dy * s * (1 + z * (1 - s))) if silu else (z, dy.copy())
    drow = np.zeros_like(row)
    for j in range(k):
        drow[j:j + steps] += w[:, j] * dz
    dw = np.stack([(dz * row[j:j + steps]).sum(0) for j in range(k)], 1)
    return dict(y=y, last=row[row.shape[0] - (k - 1):], dx=drow[k - 1:], dtaps=drow[:k - 1], dw=dw, db=dz.sum(0))


def reference(c, bounds=None, silu=True, taps=True, bias=True):
    f = {k: t.double().numpy() for k, t in c.items()}
    dim = f["x"].shape[-1]
    x, dy = f["x"].reshape(-1, dim), f["dy"].reshape(-1, dim)
    if bounds is None:
        bounds = [c["x"].shape[-2] * n for n in range(f["taps"].shape[0] + 1)]
    ref = dict(y=np.zeros_like(x), dx=np.zeros_like(x), last=np.zeros_like(f["taps"]), dtaps=np.zeros_like(f["taps"]),
               dw=np.zeros_like(f["w"]), db=np.zeros_like(f["b"]))
    for n, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        r = one(x[a:b], f["w"], f["b"] if bias else 0 * f["b"], f["taps"][n] if taps else 0 * f["taps"][n], silu, dy[a:b])
        ref["y"][a:b], ref["dx"][a:b] = r["y"], r["dx"]
        ref["last"][n], ref["dtaps"][n] = r["last"], r["dtaps"]
        ref["dw"] += r["dw"]
        ref["db"] += r["db"]
    ref["y"], ref["dx"] = ref["y"].reshape(f["x"].shape), ref["dx"].reshape(f["x"].shape)
    return ref


def check(name, got, ref):
    x = got.double().cpu().numpy()
    assert x.shape == ref.shape and np.isfinite(x).all(), name
    err = float(np.abs(x - ref).max()) / max(float(np.abs(ref).max()), 1e-30)
    assert err <= TOL[got.dtype], (name, err)


def compare(c, cu=None, bounds=None, act="silu", taps=True, bias=True):
    ref = reference(c, bounds, act == "silu", taps, bias)
    d = {k: t.cuda() for k, t in c.items()}
    tp, b = d["taps"] if taps else None, d["b"] if bias else None
    y, last = binding.conv_forward(d["x"], d["w"], b, act, tp, cu)
    g = binding.conv_backward(d["dy"], d["x"], d["w"], b, act, tp, cu)
    torch.cuda.synchronize()
    check("y", y, ref["y"])
    assert np.array_equal(last.double().cpu().numpy(), ref["last"])
    check("dx", g["dx"], ref["dx"])
    check("dw", g["dw"], ref["dw"])
    if bias:
        check("db", g["db"], ref["db"])
    else:
        assert g["db"] is None
    if taps:
        check("dtaps", g["dtaps"], ref["dtaps"])
    else:
        assert g["dtaps"] is None


@pytest.mark.parametrize("io,wt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("n,steps,dim,k", [(1, 1, 1, 4), (2, 2, 3, 4), (1, 3, 128, 4), (3, 4, 129, 3), (2, 7, 64, 2),
                                           (1, 8, 130, 4), (2, 9, 132, 4), (1, 64, 256, 4), (2, 65, 100, 3), (1, 129, 36, 2),
                                           (4, 300, 40, 4), (1, 1000, 33, 4), (300, 5, 16, 4), (9000, 3, 8, 4)])
def test_matches_float64(n, steps, dim, k, io, wt):
    compare(make((n, steps), dim, k, io, wt, 1, n))


@pytest.mark.parametrize("act,taps,bias", [("none", True, True), ("silu", False, True), ("silu", True, False),
                                           ("none", False, False)])
def test_without_activation_taps_or_bias(act, taps, bias):
    compare(make((3, 50), 64, 4, "f32", "f32", 2, 3), act=act, taps=taps, bias=bias)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,dim,k", [([5], 8, 4), ([1, 1, 1], 64, 4), ([0, 33, 0, 64, 1, 0], 70, 4),
                                           ([100, 7, 193], 96, 4), ([2, 1, 3, 2], 40, 4), ([3] * 50, 33, 3),
                                           ([0, 0, 9], 16, 2), ([500, 0, 2, 31], 128, 4)])
def test_packed_matches_float64(lengths, dim, k, io):
    bounds = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    c = make((bounds[-1],), dim, k, io, "f32", 3, len(lengths))
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    compare(c, cu, bounds)
    compare(c, cu, bounds, taps=False)


def test_steps_of_no_sequence_are_zero_and_touch_nothing():
    bounds = [13, 20, 90]
    c = make((120,), 72, 4, "bf16", "f32", 4, 2)
    for k in ("x", "dy"):
        c[k][:13] = float("nan")
        c[k][90:] = float("inf")
    clean = {k: t.clone() for k, t in c.items()}
    for k in ("x", "dy"):
        clean[k][:13] = clean[k][90:] = 0
    ref = reference(clean, bounds)
    d = {k: t.cuda() for k, t in c.items()}
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y, last = binding.conv_forward(d["x"], d["w"], d["b"], "silu", d["taps"], cu)
    g = binding.conv_backward(d["dy"], d["x"], d["w"], d["b"], "silu", d["taps"], cu)
    check("y", y, ref["y"])
    check("last", last, ref["last"])
    for k in ("dx", "dw", "db", "dtaps"):
        check(k, g[k], ref[k])
    for t in (y, g["dx"]):
        assert not t[:13].any() and not t[90:].any()


def test_a_nan_stays_in_its_sequence_and_reach():
    bounds = [0, 40, 100, 170]
    c = make((170,), 64, 4, "f32", "f32", 5, 3)
    ref = reference(c, bounds)
    c["x"][98, 7] = float("nan")
    d = {k: t.cuda() for k, t in c.items()}
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    y, _ = binding.conv_forward(d["x"], d["w"], d["b"], "silu", d["taps"], cu)
    g = binding.conv_backward(d["dy"], d["x"], d["w"], d["b"], "silu", d["taps"], cu)
    hit = torch.zeros(170, 64, dtype=torch.bool)
    hit[95:100, 7] = True
    assert y[98:100, 7].isnan().all()
    for name, t in (("y", y.cpu()), ("dx", g["dx"].cpu())):
        check(name, torch.where(hit, torch.zeros(()), t), np.where(hit.numpy(), 0, ref[name]))


def test_activation_far_from_zero():
    c = make((1, 16), 8, 4, "f32", "f32", 6, 1)
    c["x"][0, 3:6] = 300.0
    c["x"][0, 9:12] = -300.0
    compare(c)


@pytest.mark.parametrize("io,dim,wide", [("bf16", 64, 192), ("bf16", 40, 83), ("f32", 33, 70), ("f32", 64, 128)])
def test_strided_inputs(io, dim, wide):
    c = make((3, 70), dim, 4, io, "f32", 7, 3)
    d = {k: t.cuda() for k, t in c.items()}
    want = binding.conv_forward(d["x"], d["w"], d["b"], taps=d["taps"])
    back = binding.conv_backward(d["dy"], d["x"], d["w"], d["b"], taps=d["taps"])
    room = torch.full((3, 70, wide), float("nan"), dtype=d["x"].dtype, device="cuda")
    room[..., wide - dim:] = d["x"]
    x = room[..., wide - dim:]
    got = binding.conv_forward(x, d["w"], d["b"], taps=d["taps"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    again = binding.conv_backward(d["dy"], x, d["w"], d["b"], taps=d["taps"])
    assert all(torch.equal(back[k], again[k]) for k in back)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("n,steps,dim,k", [(1, 1, 64, 4), (3, 1, 33, 4), (5, 7, 100, 3), (2, 2, 4096, 4), (3, 5, 8, 2)])
def test_steps_match_whole_sequences(n, steps, dim, k, io):
    c = make((n, steps), dim, k, io, "f32", 8, n)
    ref = reference(c)
    d = {k: t.cuda() for k, t in c.items()}
    slots = torch.tensor([2 * j + 1 for j in range(n)], dtype=torch.int32, device="cuda")
    state = torch.full((2 * n + 1, k - 1, dim), 7.0, device="cuda", dtype=d["x"].dtype)
    state[slots.long()] = d["taps"]
    y = binding.conv_step(d["x"], d["w"], d["b"], state, slots)
    check("y", y, ref["y"])
    assert np.array_equal(state[slots.long()].double().cpu().numpy(), ref["last"])
    assert (state[::2] == 7).all()
    own = d["taps"].clone()
    assert torch.equal(binding.conv_step(d["x"], d["w"], d["b"], own), y)
    assert torch.equal(own, state[slots.long()])


def test_places_without_a_sequence():
    c = make((4, 2), 48, 4, "bf16", "f32", 9, 4)
    d = {k: t.cuda() for k, t in c.items()}
    state = d["taps"].clone()
    y = binding.conv_step(d["x"], d["w"], d["b"], state, torch.tensor([1, -1, 9, 0], dtype=torch.int32, device="cuda"))
    assert not y[1:3].any() and y[0].any() and y[3].any()
    assert torch.equal(state[2:], d["taps"][2:]) and not torch.equal(state[:2], d["taps"][:2])


def test_gradients_against_differences():
    c = make((1, 6), 3, 4, "f32", "f32", 10, 1)
    f = {k: t.double().numpy() for k, t in c.items()}

    def loss(**over):
        v = {**f, **over}
        return float((one(v["x"][0], v["w"], v["b"], v["taps"][0], True, f["dy"][0])["y"] * f["dy"][0]).sum())

    d = {k: t.cuda() for k, t in c.items()}
    g = binding.conv_backward(d["dy"], d["x"], d["w"], d["b"], taps=d["taps"])
    for leaf, name in (("x", "dx"), ("w", "dw"), ("b", "db"), ("taps", "dtaps")):
        num = np.zeros_like(f[leaf])
        for at in np.ndindex(num.shape):
            step = np.zeros_like(num)
            step[at] = 1e-5
            num[at] = (loss(**{leaf: f[leaf] + step}) - loss(**{leaf: f[leaf] - step})) / 2e-5
        check(name, g[name], num)


def test_same_bits_again_on_another_stream_and_in_a_graph():
    c = make((2, 300), 128, 4, "bf16", "f32", 11, 2)
    d = {k: t.cuda() for k, t in c.items()}

    def both():
        y, last = binding.conv_forward(d["x"], d["w"], d["b"], taps=d["taps"])
        return [y, last, *binding.conv_backward(d["dy"], d["x"], d["w"], d["b"], taps=d["taps"]).values()]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, last = binding.conv_forward(d["x"], d["w"], d["b"], taps=d["taps"], stream=side)
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
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn((steps, dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((dim, 4), generator=gen, device="cuda")
    cu = torch.tensor([0, steps - 100, steps], dtype=torch.int32, device="cuda")
    y, last = binding.conv_forward(x, w, cu_seqlens=cu)
    g = binding.conv_backward(x, x, w, cu_seqlens=cu)
    tail = x[steps - 100:].clone()
    y2, last2 = binding.conv_forward(tail, w)
    g2 = binding.conv_backward(tail, tail, w)
    assert torch.equal(y[steps - 100:], y2) and torch.equal(last[1:], last2) and torch.equal(g["dx"][steps - 100:], g2["dx"])
