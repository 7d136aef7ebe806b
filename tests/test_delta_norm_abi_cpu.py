"""The delta rule's and the layer norm's calls on the host: sizes, and what is refused before anything is launched.  No
GPU is needed (no call here gets past its checks)."""
import ctypes

import pytest

from selective_state_space_ssd_gb300 import binding
from selective_state_space_ssd_gb300.configs import DELTA_CONFIGS

BASE = DELTA_CONFIGS["delta_bf16"]


def delta(packed=False, **over):
    p = binding.delta_problem({**BASE, **{k: v for k, v in over.items() if k in BASE}}, packed=packed)
    for k, v in over.items():
        if k not in BASE:
            setattr(p, k, v)
    return p


def stash_status(lib, p):
    n = ctypes.c_size_t(0)
    return lib.ssd_delta_stash_size(ctypes.byref(p) if p is not None else None, ctypes.byref(n))


@pytest.mark.parametrize("over,code", [
    (dict(), 0), (dict(key_dim=1, value_dim=1), 0), (dict(seqlen=1), 0), (dict(gate_dtype="bf16"), 0),
    (dict(q_stride=8 * 128), 0), (dict(q_stride=8 * 128 + 3), 0),
    (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(nheads=0), 1), (dict(value_heads=0), 1), (dict(key_dim=0), 1),
    (dict(value_dim=-1), 1), (dict(packed=2), 1), (dict(io_dtype=5), 1), (dict(gate_dtype=7), 1), (dict(k_stride=-1), 1),
    (dict(value_heads=12), 2), (dict(key_dim=129), 2), (dict(value_dim=129), 2), (dict(q_stride=8 * 128 - 1), 2),
    (dict(v_stride=100), 2), (dict(seqlen=1 << 31), 2), (dict(batch=1 << 20, seqlen=1 << 12), 2),
    (dict(nheads=1, value_heads=65536), 2), (dict(dtype="f32"), 3),
])
def test_delta_problem_checks(cuda_lib, over, code):
    if isinstance(over.get("gate_dtype"), int):
        p = delta()
        p.gate_dtype = over["gate_dtype"]
    else:
        p = delta(**over)
    assert stash_status(cuda_lib, p) == code


def test_delta_sizes(cuda_lib):
    assert stash_status(cuda_lib, None) == 1
    assert cuda_lib.ssd_delta_stash_size(ctypes.byref(delta()), None) == 1
    items = 2 * 16 * 16  # sequences x chunks x value heads
    per = 128 * 128 * 2 + 64 * 128 * 2 + 34048
    got = binding.ssd_delta_stash_size(delta())
    assert items * per <= got <= items * per + 2048
    fwd, bwd = (binding.ssd_delta_workspace_size(delta(), b) for b in (False, True))
    fwd_s, bwd_s = (binding.ssd_delta_workspace_size(delta(), b, True) for b in (False, True))
    assert fwd_s >= 256 and bwd_s < bwd and fwd_s < fwd < bwd
    assert fwd - fwd_s >= items * 34048  # the stash holds the chunk records
    # a packed batch may end a chunk early in every sequence
    p = delta(packed=True, batch=5, seqlen=100)
    assert binding.ssd_delta_stash_size(p) >= (100 // 64 + 5) * 16 * per


def test_delta_calls_refuse_bad_pointers(cuda_lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("uses fake device addresses; host-only check")
    f = 1 << 20  # never dereferenced
    p, big = delta(), 1 << 40
    call = lambda p=p, q=f, k=f, v=f, g=f, beta=f, s0=None, cu=None, o=f, sf=f, stash=None, sb=0, ws=f, nb=big: (  # noqa: E731
        cuda_lib.ssd_delta_forward(ctypes.byref(p), q, k, v, g, beta, s0, cu, 1.0, o, sf, stash, sb, ws, nb, None))
    for name in ("q", "k", "v", "g", "beta", "o", "ws"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "k", "v"):
        assert call(**{name: f + 1}) == 4, name
    for name in ("g", "beta", "o", "ws", "s0", "sf"):
        assert call(**{name: f + 8}) == 4, name
    assert call(cu=f) == 1 and call(p=delta(packed=True)) == 1 and call(p=delta(packed=True), cu=f + 2) == 4
    assert call(nb=binding.ssd_delta_workspace_size(p, False) - 1) == 5
    assert call(stash=f, sb=binding.ssd_delta_stash_size(p) - 1) == 5 and call(stash=f + 8, sb=big) == 4
    back = lambda **o: cuda_lib.ssd_delta_backward(ctypes.byref(p), *(o.get(n, f) for n in (  # noqa: E731
        "dout", "ds", "q", "k", "v", "g", "beta")), None, None, 1.0, *(o.get(n, f) for n in (
            "dq", "dk", "dv", "dg", "dbeta")), o.get("ds0"), None, 0, o.get("ws", f), o.get("nb", big), None)
    for name in ("dout", "q", "k", "v", "g", "beta", "dq", "dk", "dv", "dg", "dbeta", "ws"):
        assert back(**{name: None}) == 1, name
    assert back(dq=f + 8) == 4 and back(ds=f + 4) == 4 and back(ds0=f + 8) == 4 and back(q=f + 1) == 4
    assert back(nb=binding.ssd_delta_workspace_size(p, True) - 1) == 5
    step = lambda p=p, state=f, slots=None, n=2, o=f, q=f: cuda_lib.ssd_delta_step(  # noqa: E731
        ctypes.byref(p), q, f, f, f, f, state, slots, n, 1.0, o, None)
    assert step(state=None) == 1 and step(o=None) == 1 and step(q=None) == 1 and step(n=0) == 1
    assert step(n=1) == 1  # fewer slots than sequences, and no slot numbers
    assert step(p=delta(packed=True)) == 1 and step(state=f + 8) == 4 and step(slots=f + 2) == 4 and step(q=f + 1) == 4
    assert step(p=delta(dtype="f32"), q=f + 2) == 4  # fp32 is taken here, on its own alignment


def norm(**over):
    p = binding.ssd_norm_problem(1, 0, 10, 100, 0)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,code", [
    (dict(), 0), (dict(dim=16384), 0), (dict(dim=1, rows=1), 0), (dict(x_stride=101), 0),
    (dict(rows=0), 1), (dict(dim=0), 1), (dict(io_dtype=2), 1), (dict(weight_dtype=-1), 1), (dict(x_stride=-1), 1),
    (dict(dim=16385), 2), (dict(rows=1 << 31), 2), (dict(x_stride=99), 2),
])
def test_norm_problem_checks(cuda_lib, over, code):
    n = ctypes.c_size_t(0)
    assert cuda_lib.ssd_norm_workspace_size(ctypes.byref(norm(**over)), ctypes.byref(n)) == code
    assert (n.value >= 256) == (code == 0)


def test_norm_calls_refuse_bad_pointers(cuda_lib):
    import torch
    n = ctypes.c_size_t(0)
    assert cuda_lib.ssd_norm_workspace_size(None, ctypes.byref(n)) == 1
    assert cuda_lib.ssd_norm_workspace_size(ctypes.byref(norm()), None) == 1
    if torch.cuda.is_available():
        pytest.skip("uses fake device addresses; host-only check")
    f, p = 1 << 20, norm()
    fwd = lambda x=f, w=f, b=f, eps=1e-5, y=f, m=f, r=f: cuda_lib.ssd_norm_forward(  # noqa: E731
        ctypes.byref(p), x, w, b, eps, y, m, r, None)
    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1
    assert fwd(x=f + 1) == 4 and fwd(w=f + 8) == 4 and fwd(b=f + 8) == 4 and fwd(y=f + 8) == 4 and fwd(m=f + 2) == 4
    bwd = lambda dy=f, x=f, m=f, r=f, dx=f, dw=f, db=f, ws=f, nb=1 << 30: cuda_lib.ssd_norm_backward(  # noqa: E731
        ctypes.byref(p), dy, x, m, r, f, dx, dw, db, ws, nb, None)
    for name in ("dy", "x", "m", "r", "dx", "ws"):
        assert bwd(**{name: None}) == 1, name
    assert bwd(dx=f + 8) == 4 and bwd(dw=f + 4) == 4 and bwd(r=f + 1) == 4
    assert bwd(nb=binding.ssd_norm_workspace_size(p) - 1) == 5
