"""GPU parity of the gated delta rule with one decay per head (through the C ABI) with the float64 recurrence of
oracle/kda.py, which is the same rule with one decay per key row.

Bounds (max|gpu - ref| / max|ref|), set from the arithmetic before the first run:

* s_final: what the state's products drop is 2^-17 of each factor, a few factors deep: 3e-5 (4 x 2^-17).
* o: one rounding to bf16 (2^-9) and the scores' rounding (2^-9 of each term): 8e-3 (4 x 2^-9).
* ds0: the scores' rounding, through dR: 8e-3.
* the other gradients: three bf16 tiles deep and rounded: the library's bf16 bound, 2e-2.
* the step form: fp32 arithmetic, 1e-5 for the state and for fp32 o; bf16 o one rounding, 4e-3 (2 x 2^-9).
"""
import numpy as np
import pytest
import torch

from oracle.kda import kda_backward, kda_forward
from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu

TOL_F = {"o": 8e-3, "s_final": 3e-5}
TOL_B = {"dq": 2e-2, "dk": 2e-2, "dv": 2e-2, "dg": 2e-2, "dbeta": 2e-2, "ds0": 8e-3}


def cfg_of(b=1, T=64, H=1, HV=1, K=16, V=16, gates="f32", dtype="bf16"):
    return dict(dtype=dtype, gate_dtype=gates, batch=b, seqlen=T, nheads=H, value_heads=HV, key_dim=K, value_dim=V)


def make(cfg, seed, packed=False, decay=0.3, corr=0.3):
    """Seeded CPU inputs: unit keys of mostly one sign (corr: how far their mean is from zero), beta in (0, 1), g from
    -decay down by head, do and ds_final ~ N(0, 1)."""
    gen = torch.Generator().manual_seed(seed)
    b, T, H, HV, K, V = (cfg[n] for n in ("batch", "seqlen", "nheads", "value_heads", "key_dim", "value_dim"))
    lead = (1, T) if packed else (b, T)
    io = {"bf16": torch.bfloat16, "f32": torch.float32}[cfg["dtype"]]
    gt = {"bf16": torch.bfloat16, "f32": torch.float32}[cfg["gate_dtype"]]
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    out = dict(q=unit(rn(*lead, H, K) + corr), k=unit(rn(*lead, H, K) + corr), v=rn(*lead, HV, V), do=rn(*lead, HV, V))
    out = {n: x.to(io) for n, x in out.items()}
    out["g"] = (-decay * torch.rand((*lead, HV), generator=gen) * (1 + torch.arange(HV))).to(gt)
    out["beta"] = torch.rand((*lead, HV), generator=gen).to(gt)
    out["s0"] = 0.5 * rn(b, HV, K, V)
    out["ds_final"] = rn(b, HV, K, V)
    return out


def f64(x):
    return {n: (None if t is None else t.double().numpy()) for n, t in x.items()}


def oracle(cfg, cpu, scale, s0=True, ds_final=True, backward=True):
    """o, s_final and the gradients of <do, o> + <ds_final, s_final> in float64."""
    f = f64(cpu)
    K = cfg["key_dim"]
    g = np.repeat(f["g"][..., None], K, axis=-1)
    z = f["s0"] if s0 else np.zeros_like(f["s0"])
    out = dict(kda_forward(f["q"], f["k"], f["v"], g, f["beta"], z, scale))
    if backward:
        ds = f["ds_final"] if ds_final else np.zeros_like(f["ds_final"])
        out.update(kda_backward(f["do"], ds, f["q"], f["k"], f["v"], g, f["beta"], z, scale))
        out["dg"] = out["dg"].sum(-1)
    return out


def run(cfg, dev, scale=None, s0=True, ds_final=True, cu=None, stash=None, backward=True):
    x = tuple(dev[n] for n in ("q", "k", "v", "g", "beta"))
    z = dev["s0"] if s0 else None
    o, sf = binding.delta_forward(cfg, *x, s0=z, scale=scale, cu_seqlens=cu, stash=stash)
    out = dict(o=o, s_final=sf)
    if backward:
        out.update(binding.delta_backward(cfg, dev["do"], *x, ds_final=dev["ds_final"] if ds_final else None, s0=z,
                                          scale=scale, cu_seqlens=cu, stash=stash))
    torch.cuda.synchronize()
    return out


def cuda(cpu):
    return {n: t.cuda() for n, t in cpu.items()}


def rel(got, ref):
    x = got.detach().double().cpu().numpy()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert np.isfinite(x).all()
    return float(np.abs(x - ref).max()) / max(float(np.abs(ref).max()), 1e-30)


def check(got, ref, tols):
    errs = {n: rel(got[n], ref[n]) for n in tols if got.get(n) is not None}
    assert all(errs[n] <= tols[n] for n in errs), errs
    return errs


CASES = {
    "one_step": cfg_of(b=2, T=1, H=2, HV=4, K=8, V=8),
    "two_steps": cfg_of(T=2, K=5, V=3),
    "one_chunk": cfg_of(T=64, K=64, V=32),
    "chunk_and_one": cfg_of(T=65, H=1, HV=2, K=128, V=16),
    "chunk_less_one": cfg_of(T=63, K=128, V=128, gates="bf16"),
    "ragged": cfg_of(b=3, T=150, H=2, HV=4, K=37, V=45),
    "even_unaligned": cfg_of(b=2, T=70, H=1, HV=3, K=66, V=100),
    "narrow_v": cfg_of(T=130, H=2, HV=2, K=96, V=1),
    "narrow_k": cfg_of(T=130, H=2, HV=2, K=1, V=24, gates="bf16"),
    "grouped": cfg_of(b=2, T=100, H=2, HV=8, K=72, V=40),
    "dim128": cfg_of(b=2, T=300, H=2, HV=4, K=128, V=128, gates="bf16"),
}

# chunk counts at which a scan of few heads is cut into runs, and at which a block takes several chunks in turn
LONG = {
    "few_heads": cfg_of(T=64 * 40 + 7, H=1, HV=2, K=40, V=72),
    "one_head": cfg_of(T=64 * 33, H=1, HV=1, K=128, V=128, gates="bf16"),
    "unaligned": cfg_of(b=2, T=64 * 24 + 1, H=1, HV=1, K=33, V=17),
    "many_chunks": cfg_of(b=3, T=64 * 20 + 5, H=3, HV=9, K=16, V=16),
}


@pytest.mark.parametrize("name", sorted(LONG))
def test_long_sequences_match_the_oracle(name):
    cfg = LONG[name]
    cpu = make(cfg, 14, decay=0.01)
    got = run(cfg, cuda(cpu))
    check(got, oracle(cfg, cpu, cfg["key_dim"] ** -0.5), {**TOL_F, **TOL_B})
    again = run(cfg, cuda(cpu), stash=binding.delta_stash(cfg))
    for k in got:
        assert torch.equal(got[k], again[k]), k


def test_long_packed_sequences_match_the_oracle():
    """Two long sequences, short ones and empty ones in one batch, cut into runs by their mean length."""
    lengths = [64 * 37 + 3, 0, 64 * 70, 5, 0]
    cfg = cfg_of(b=5, T=sum(lengths), H=1, HV=1, K=32, V=24)
    cpu = make(cfg, 15, packed=True, decay=0.01)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    got = run(cfg, cuda(cpu), cu=cu.cuda())
    for i, (a, length) in enumerate(zip(cu[:-1].tolist(), lengths)):
        if not length:
            assert torch.equal(got["s_final"][i].cpu(), cpu["s0"][i]) and torch.equal(got["ds0"][i].cpu(), cpu["ds_final"][i])
            continue
        one = {k: (x[i:i + 1] if k in ("s0", "ds_final") else x[:, a:a + length]) for k, x in cpu.items()}
        ref = oracle(dict(cfg, batch=1, seqlen=length), one, 32 ** -0.5)
        part = {k: (x[i:i + 1] if k in ("s_final", "ds0") else x[:, a:a + length]) for k, x in got.items()}
        check(part, ref, {**TOL_F, **TOL_B})


def test_more_sequences_than_are_ranked():
    """Up to 1024 packed sequences are taken by length, more in their order: the same results bit for bit."""
    lengths = [(7 * i) % 5 + 70 * (i % 11 == 3) for i in range(1300)]
    cfg = cfg_of(b=1300, T=sum(lengths), H=1, HV=2, K=16, V=16)
    dev = cuda(make(cfg, 17, packed=True))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    got = run(cfg, dev, cu=cu.cuda())
    for a, b in ((0, 1024), (900, 1300)):
        t0, t1 = int(cu[a]), int(cu[b])
        part = {k: (x[a:b] if k in ("s0", "ds_final") else x[:, t0:t1]).contiguous() for k, x in dev.items()}
        alone = run(dict(cfg, batch=b - a, seqlen=t1 - t0), part, cu=(cu[a:b + 1] - t0).cuda())
        for k, x in alone.items():
            assert torch.equal(x, got[k][a:b] if k in ("s_final", "ds0") else got[k][:, t0:t1]), k


@pytest.mark.parametrize("name", sorted(CASES))
def test_matches_the_oracle(name):
    cfg = CASES[name]
    cpu = make(cfg, 1)
    scale = cfg["key_dim"] ** -0.5
    check(run(cfg, cuda(cpu)), oracle(cfg, cpu, scale), {**TOL_F, **TOL_B})


def test_no_initial_state_no_final_gradient():
    cfg = CASES["ragged"]
    cpu = make(cfg, 2)
    got = run(cfg, cuda(cpu), scale=0.7, s0=False, ds_final=False)
    assert got["ds0"] is None
    check(got, oracle(cfg, cpu, 0.7, s0=False, ds_final=False), {**TOL_F, **TOL_B})


@pytest.mark.parametrize("decay,corr", [(0.0, 0.3), (0.002, 0.3), (3.0, 0.3), (30.0, 0.3), (0.05, 3.0)])
def test_decays_and_correlated_keys(decay, corr):
    """No decay, slow, fast and vanishing decays; keys that nearly point one way (the inverse's hard case)."""
    cfg = cfg_of(b=1, T=200, H=1, HV=2, K=64, V=32)
    cpu = make(cfg, 3, decay=decay, corr=corr)
    check(run(cfg, cuda(cpu)), oracle(cfg, cpu, 0.125), {**TOL_F, **TOL_B})


def test_a_gate_of_minus_infinity_forgets_the_state():
    cfg = cfg_of(b=1, T=100, H=1, HV=1, K=32, V=16)
    cpu = make(cfg, 4)
    for t in (0, 17, 64, 99):
        cpu["g"][0, t, 0] = -float("inf")
    ref_in = dict(cpu, g=cpu["g"].clamp_min(-2000.0))  # exp(-2000) is 0 in float64 too
    check(run(cfg, cuda(cpu)), oracle(cfg, ref_in, 32 ** -0.5), {**TOL_F, **TOL_B})


LENGTHS = {
    "some_empty": [0, 70, 0, 0, 1, 64, 129, 3, 0],
    "one": [200],
    "all_short": [1, 2, 3, 1, 1, 5],
    "many": [(i * 37) % 23 for i in range(1100)],
    "all_empty_but_one_step": [0, 0, 1, 0],
}


@pytest.mark.parametrize("name", sorted(LENGTHS))
def test_packed_sequences_are_sequences_by_themselves(name):
    lengths = LENGTHS[name]
    T, n = sum(lengths), len(lengths)
    cfg = cfg_of(b=n, T=T, H=1, HV=2, K=24, V=20)
    cpu = make(cfg, 5, packed=True)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    got = run(cfg, cuda(cpu), cu=cu.cuda())
    scale = 24 ** -0.5
    ref = {k: np.zeros(tuple(got[k].shape)) for k in {**TOL_F, **TOL_B}}
    for i, (a, length) in enumerate(zip(cu[:-1].tolist(), lengths)):
        ref["s_final"][i] = cpu["s0"][i].numpy()
        ref["ds0"][i] = cpu["ds_final"][i].numpy()
        if not length:
            continue
        one = {k: (x[i:i + 1] if k in ("s0", "ds_final") else x[:, a:a + length]) for k, x in cpu.items()}
        r = oracle(dict(cfg, batch=1, seqlen=length), one, scale)
        for k in ref:
            if k in ("s_final", "ds0"):
                ref[k][i] = r[k][0]
            else:
                ref[k][:, a:a + length] = r[k]
    check(got, ref, {**TOL_F, **TOL_B})
    if name != "many":  # empty sequences: bit for bit
        for i, length in enumerate(lengths):
            if not length:
                assert torch.equal(got["s_final"][i].cpu(), cpu["s0"][i])
                assert torch.equal(got["ds0"][i].cpu(), cpu["ds_final"][i])


def test_bad_bounds_are_pulled_in():
    """cu_seqlens that leave the axis or run backwards: every access stays inside, steps of real sequences are right."""
    cfg = cfg_of(b=3, T=100, H=1, HV=1, K=16, V=16)
    cpu = make(cfg, 6, packed=True)
    cu = torch.tensor([0, 60, 20, 1000], dtype=torch.int32).cuda()  # 60, 0 and 40 steps
    good = torch.tensor([0, 60, 60, 100], dtype=torch.int32).cuda()
    a, b = run(cfg, cuda(cpu), cu=cu), run(cfg, cuda(cpu), cu=good)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_tensors_inside_wider_ones():
    """q, k, v as slices of one projection (strided, and starting off 16 bytes) give the bits of dense ones."""
    cfg = cfg_of(b=2, T=90, H=2, HV=4, K=32, V=24)
    cpu = make(cfg, 7)
    dense = run(cfg, cuda(cpu))
    for pad in (8, 1):
        wide = torch.full((2, 90, pad + 64 + 64 + 96 + 3 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        x = cuda(cpu)
        at = pad
        for n, w in (("q", 64), ("k", 64), ("v", 96)):
            part = wide[:, :, at:at + w]
            part.copy_(x[n].reshape(2, 90, w))
            x[n] = part.unflatten(2, (-1, 32 if n != "v" else 24))
            at += w
        got = run(cfg, x)
        for k in dense:
            assert torch.equal(got[k], dense[k]), (pad, k)


def test_stash_gives_the_bits_of_the_recompute_and_calls_repeat():
    for cfg, packed in ((CASES["dim128"], False), (CASES["ragged"], False), (cfg_of(b=4, T=333, HV=2, K=64, V=64), True)):
        cpu = make(cfg, 8, packed=packed)
        dev = cuda(cpu)
        cu = torch.tensor([0, 100, 100, 101, 333], dtype=torch.int32, device="cuda") if packed else None
        stash = binding.delta_stash(cfg, packed=packed)
        stash.fill_(255)  # NaN everywhere that the forward does not fill
        a, b, c = run(cfg, dev, cu=cu), run(cfg, dev, cu=cu), run(cfg, dev, cu=cu, stash=stash)
        for k in a:
            assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


def test_a_workspace_full_of_nan_changes_nothing():
    cfg = cfg_of(b=2, T=77, H=1, HV=2, K=40, V=24)
    dev = cuda(make(cfg, 9))
    x = tuple(dev[n] for n in ("q", "k", "v", "g", "beta"))
    plain = run(cfg, dev)
    prob = binding.delta_problem(cfg)
    wf, wb = (torch.full((binding.ssd_delta_workspace_size(prob, b),), 255, dtype=torch.uint8, device="cuda") for b in (False, True))
    o, sf = binding.delta_forward(cfg, *x, s0=dev["s0"], workspace=(wf, wf.numel()))
    g = binding.delta_backward(cfg, dev["do"], *x, ds_final=dev["ds_final"], s0=dev["s0"], workspace=(wb, wb.numel()))
    torch.cuda.synchronize()
    for k, t in dict(g, o=o, s_final=sf).items():
        assert torch.equal(t, plain[k]), k
    assert int(wf[:4].view(torch.int32)) == 0 and int(wb[:4].view(torch.int32)) == 0


def test_other_sequences_take_nothing_from_a_nan():
    cfg = cfg_of(b=3, T=100, H=1, HV=2, K=32, V=32)
    cpu = make(cfg, 10)
    clean = run(cfg, cuda(cpu))
    cpu["v"][1, 50] = float("nan")
    cpu["k"][1, 70] = float("inf")
    got = run(cfg, cuda(cpu))
    for k in ("o", "s_final", "dq", "dk", "dv", "dg", "dbeta", "ds0"):
        for n in (0, 2):
            assert torch.equal(got[k][n], clean[k][n]), (k, n)
    assert got["o"][1].isnan().any()


def test_a_sequence_in_pieces_is_the_whole():
    cfg = cfg_of(b=2, T=200, H=1, HV=2, K=64, V=48)
    cpu = make(cfg, 11)
    dev = cuda(cpu)
    whole = run(cfg, dev, backward=False)
    s, parts = dev["s0"], []
    for a, b in ((0, 77), (77, 78), (78, 200)):
        piece = {n: dev[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")}
        o, s = binding.delta_forward(dict(cfg, seqlen=b - a), *piece.values(), s0=s)
        parts.append(o)
    assert rel(torch.cat(parts, 1), whole["o"].double().cpu().numpy()) <= 8e-3
    assert rel(s, whole["s_final"].double().cpu().numpy()) <= 6e-5


def test_gradients_against_differences():
    """Directional derivatives of the float64 loss, by central differences, against the kernels' gradients."""
    cfg = cfg_of(b=1, T=80, H=1, HV=2, K=16, V=12)
    cpu = make(cfg, 12)
    got = run(cfg, cuda(cpu))
    f = f64(cpu)

    def loss(x):
        g = np.repeat(x["g"][..., None], 16, axis=-1)
        r = kda_forward(x["q"], x["k"], x["v"], g, x["beta"], x["s0"], 0.25)
        return float((f["do"] * r["o"]).sum() + (f["ds_final"] * r["s_final"]).sum())

    for n in ("q", "k", "v", "g", "beta", "s0"):
        grad = got["d" + n].double().cpu().numpy()
        way = grad / np.linalg.norm(grad)  # along the gradient itself: the derivative is its length
        h = 1e-5
        fd = (loss(dict(f, **{n: f[n] + h * way})) - loss(dict(f, **{n: f[n] - h * way}))) / (2 * h)
        assert abs(fd - np.linalg.norm(grad)) <= 1e-2 * abs(fd), (n, fd, np.linalg.norm(grad))


def test_on_a_side_stream():
    cfg = CASES["dim128"]
    dev = cuda(make(cfg, 13))
    ref = run(cfg, dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run(cfg, dev)
    st.synchronize()
    for k in ref:
        assert torch.equal(ref[k], got[k]), k


def test_offsets_past_32_bits():
    """More than 2^31 elements of v and o: the last chunks are those of a short run (the state is empty until then)."""
    hv, tail, T = 64, 100, 64 * 4099 + 1
    cfg = cfg_of(T=T, H=1, HV=hv, K=16, V=128)
    assert T * hv * 128 > 1 << 31
    short = cuda(make(cfg_of(T=tail, H=1, HV=hv, K=16, V=128), 16))
    x = dict(q=torch.zeros((1, T, 1, 16), dtype=torch.bfloat16, device="cuda"))
    x["k"] = torch.zeros_like(x["q"])
    x["v"] = torch.zeros((1, T, hv, 128), dtype=torch.bfloat16, device="cuda")
    x["g"] = torch.zeros((1, T, hv), device="cuda")
    x["beta"] = torch.zeros_like(x["g"])
    for n in x:
        x[n][:, -tail:] = short[n]
    o, sf = binding.delta_forward(cfg, *x.values())
    want_o, want_sf = binding.delta_forward(dict(cfg, seqlen=tail), *(short[n] for n in x))
    assert (o[:, :-tail] == 0).all()
    assert rel(o[:, -tail:], want_o.double().cpu().numpy()) <= 8e-3  # (other chunk bounds, other roundings)
    assert rel(sf, want_sf.double().cpu().numpy()) <= 6e-5


# ---------------------------------------------------------------- the step form
STEP_CASES = {
    "one": (cfg_of(b=1, T=1, H=1, HV=2, K=128, V=128), 1),
    "batch": (cfg_of(b=5, T=1, H=2, HV=4, K=128, V=128, gates="bf16"), 9),
    "draft": (cfg_of(b=3, T=5, H=2, HV=2, K=64, V=32), 3),
    "ragged": (cfg_of(b=3, T=4, H=1, HV=3, K=37, V=45), 7),
    "narrow": (cfg_of(b=2, T=3, H=1, HV=1, K=1, V=1), 2),
    "f32": (cfg_of(b=4, T=7, H=2, HV=4, K=96, V=100, dtype="f32"), 6),
    "f32_ragged": (cfg_of(b=2, T=2, H=1, HV=1, K=65, V=33, dtype="f32", gates="bf16"), 2),
}


@pytest.mark.parametrize("name", sorted(STEP_CASES))
def test_step_matches_the_oracle(name):
    cfg, slots = STEP_CASES[name]
    b = cfg["batch"]
    cpu = make(cfg, 21)
    gen = torch.Generator().manual_seed(22)
    cache = torch.randn((slots, cfg["value_heads"], cfg["key_dim"], cfg["value_dim"]), generator=gen)
    at = torch.randperm(slots, generator=gen)[:b].to(torch.int32)
    ref = oracle(cfg, dict(cpu, s0=cache[at.long()]), 0.3, backward=False)
    state = cache.cuda()
    dev = cuda(cpu)
    o = binding.delta_step(cfg, *(dev[n] for n in ("q", "k", "v", "g", "beta")), state, at.cuda(), 0.3)
    torch.cuda.synchronize()
    assert rel(o, ref["o"]) <= (1e-5 if cfg["dtype"] == "f32" else 4e-3)
    assert rel(state[at.long().cuda()], ref["s_final"]) <= 1e-5
    rest = [i for i in range(slots) if i not in at.tolist()]
    assert torch.equal(state[rest].cpu(), cache[rest])  # the other slots are untouched


def test_step_slots_past_32_bits():
    """A cache of more than 2^31 elements: the last slots are the sequences' own."""
    cfg = cfg_of(b=2, T=2, H=8, HV=32, K=128, V=128)
    dev = cuda(make(cfg, 26))
    x = tuple(dev[n] for n in ("q", "k", "v", "g", "beta"))
    slots = (1 << 31) // (32 * 128 * 128) + 3
    state = torch.empty((slots, 32, 128, 128), device="cuda")
    at = torch.tensor([slots - 1, slots - 2], dtype=torch.int32, device="cuda")
    state[at.long()] = dev["s0"]
    o = binding.delta_step(cfg, *x, state, at)
    want = dev["s0"].clone()
    assert torch.equal(o, binding.delta_step(cfg, *x, want)) and torch.equal(state[at.long()], want)


def test_step_places_without_a_sequence():
    cfg = cfg_of(b=5, T=2, H=1, HV=2, K=32, V=20)
    dev = cuda(make(cfg, 23))
    x = tuple(dev[n] for n in ("q", "k", "v", "g", "beta"))
    cache = torch.randn((4, 2, 32, 20), generator=torch.Generator().manual_seed(1)).cuda()
    state = cache.clone()
    slots = torch.tensor([2, -1, 4, 0, 1 << 30], dtype=torch.int32, device="cuda")
    o = binding.delta_step(cfg, *x, state, slots)
    assert (o[[1, 2, 4]] == 0).all() and torch.equal(state[[1, 3]], cache[[1, 3]])
    alone = cache.clone()
    one = tuple(t[[0, 3]].contiguous() for t in x)
    o2 = binding.delta_step(dict(cfg, batch=2), *one, alone, torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(o[[0, 3]], o2) and torch.equal(state, alone)


def test_steps_continue_a_prompt():
    """A prompt by chunks and then token by token is the whole sequence by chunks."""
    cfg = cfg_of(b=2, T=140, H=2, HV=4, K=64, V=64)
    cpu = make(cfg, 24)
    ref = oracle(cfg, cpu, 0.125, backward=False)
    dev = cuda(cpu)
    x = {n: dev[n] for n in ("q", "k", "v", "g", "beta")}
    o, state = binding.delta_forward(dict(cfg, seqlen=130), *(t[:, :130].contiguous() for t in x.values()), s0=dev["s0"])
    outs = [o]
    for t in range(130, 140):
        outs.append(binding.delta_step(dict(cfg, seqlen=1), *(y[:, t:t + 1].contiguous() for y in x.values()), state))
    assert rel(torch.cat(outs, 1), ref["o"]) <= 8e-3
    assert rel(state, ref["s_final"]) <= 3e-5


def test_step_in_a_graph():
    cfg = cfg_of(b=4, T=1, H=1, HV=2, K=128, V=64)
    dev = cuda(make(cfg, 25))
    x = tuple(dev[n] for n in ("q", "k", "v", "g", "beta"))
    state = dev["s0"].clone()
    want = state.clone()
    for _ in range(3):
        o_want = binding.delta_step(cfg, *x, want)
    binding.delta_step(cfg, *x, state.clone())  # loads the module before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = binding.delta_step(cfg, *x, state)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, want) and torch.equal(o, o_want)


# ---------------------------------------------------------------- refusals
def test_refusals():
    cfg = cfg_of(b=1, T=8, H=2, HV=4, K=16, V=16)
    dev = cuda(make(cfg, 31))
    x = {n: dev[n] for n in ("q", "k", "v", "g", "beta")}
    call = lambda c=cfg, **o: binding.delta_forward(c, *dict(x, **o).values())  # noqa: E731
    call()
    for bad in (dict(q=x["q"].float()), dict(k=x["k"][..., :8]), dict(v=x["v"].transpose(1, 2)), dict(g=x["g"].bfloat16()),
                dict(beta=x["beta"][:, :4])):
        with pytest.raises(ValueError):
            call(**bad)
    status = lambda c: _status(lambda: binding.delta_stash(c))  # noqa: E731
    assert status(dict(cfg, value_heads=3)) == 2 and status(dict(cfg, key_dim=129)) == 2
    assert status(dict(cfg, value_dim=129)) == 2 and status(dict(cfg, seqlen=0)) == 1
    assert status(dict(cfg, dtype="f32")) == 3
    prob = binding.delta_problem(cfg)
    o, sf = torch.empty_like(x["v"]), torch.empty_like(dev["s0"])
    n = binding.ssd_delta_workspace_size(prob, False)
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
    raw = lambda p=prob, cu=None, oo=o, w=ws, nb=n, stash=None, sb=0, q=x["q"]: _status(  # noqa: E731
        lambda: binding.ssd_delta_forward(p, q, x["k"], x["v"], x["g"], x["beta"], None, cu, 1.0, oo, sf, stash, sb, w, nb))
    assert raw() == 0
    assert raw(nb=n - 1) == 5 and raw(w=None) == 1 and raw(oo=None) == 1 and raw(q=None) == 1
    assert raw(w=ws.data_ptr() + 8) == 4 and raw(q=x["q"].data_ptr() + 1) == 4
    assert raw(cu=torch.zeros(2, dtype=torch.int32, device="cuda")) == 1  # bounds for a problem that is not packed
    assert raw(p=binding.delta_problem(cfg, packed=True)) == 1            # and the other way round
    need = binding.ssd_delta_stash_size(prob)
    assert raw(stash=torch.empty(need, dtype=torch.uint8, device="cuda"), sb=need - 1) == 5
    short = binding.delta_problem(cfg)
    short.q_stride = 31
    assert raw(p=short) == 2
    short.q_stride = -1
    assert raw(p=short) == 1
    state = torch.zeros((1, 4, 16, 16), device="cuda")
    step = lambda p=prob, s=state, slots=None, k=1: _status(  # noqa: E731
        lambda: binding.ssd_delta_step(p, x["q"], x["k"], x["v"], x["g"], x["beta"], s, slots, k, 1.0, o))
    assert step() == 0 and step(k=0) == 1 and step(s=None) == 1 and step(s=state.data_ptr() + 4) == 4
    assert step(p=binding.delta_problem(cfg, packed=True)) == 1
    torch.cuda.synchronize()


def _status(f):
    try:
        f()
    except binding.SSDError as e:
        return e.status
    return 0
