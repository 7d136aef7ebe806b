"""The recurrence's, the convolution's and the feed-forward's calls on the host: sizes, and what is refused before anything
is launched.  No GPU is needed (no call here gets past its checks)."""
import ctypes

import pytest
import torch

from selective_state_space_ssd_gb300 import binding


def struct(kind, **over):
    p = {"glr": lambda: binding.ssd_glr_problem(1, 0, 2, 100, 48, 0, 0, 0),
         "conv": lambda: binding.ssd_conv_problem(1, 0, 0, 1, 2, 100, 48, 4, 0),
         "ffn": lambda: binding.ssd_ffn_problem(1, 1, 100, 48, 96, 0)}[kind]()
    for k, v in over.items():
        setattr(p, k, v)
    return p


def size_status(lib, kind, p):
    n = ctypes.c_size_t(0)
    ref = None if p is None else ctypes.byref(p)
    call = {"glr": lambda out: lib.ssd_glr_workspace_size(ref, 0, out), "conv": lambda out: lib.ssd_conv_workspace_size(ref, out),
            "ffn": lambda out: lib.ssd_ffn_workspace_size(ref, 1, 0, out)}[kind]
    assert call(None) == 1
    code = call(ctypes.byref(n))
    assert (n.value >= 256) == (code == 0)
    return code


@pytest.mark.parametrize("kind,over,code", [
    ("glr", dict(), 0), ("glr", dict(io_dtype=0), 0), ("glr", dict(dim=1, seqlen=1, batch=1), 0), ("glr", dict(x_stride=49), 0),
    ("glr", dict(packed=1, batch=1 << 20, seqlen=5), 0), ("glr", dict(dim=1 << 24), 0),
    ("glr", dict(batch=0), 1), ("glr", dict(seqlen=0), 1), ("glr", dict(dim=0), 1), ("glr", dict(io_dtype=2), 1),
    ("glr", dict(packed=2), 1), ("glr", dict(r_stride=-1), 1), ("glr", dict(i_stride=47), 2), ("glr", dict(batch=65536), 2),
    ("glr", dict(seqlen=1 << 31), 2), ("glr", dict(batch=1 << 12, seqlen=1 << 20), 2), ("glr", dict(dim=(1 << 24) + 1), 2),
    ("glr", dict(x_stride=(1 << 24) + 1), 2), ("glr", dict(packed=1, batch=1 << 29), 2),
    ("conv", dict(), 0), ("conv", dict(taps=2, weight_dtype=1), 0), ("conv", dict(activation=0, io_dtype=0), 0),
    ("conv", dict(taps=0), 1), ("conv", dict(activation=2), 1), ("conv", dict(weight_dtype=3), 1), ("conv", dict(packed=-1), 1),
    ("conv", dict(taps=1), 2), ("conv", dict(taps=5), 2), ("conv", dict(x_stride=47), 2), ("conv", dict(batch=65536), 2),
    ("conv", dict(dim=(1 << 20) + 1), 2), ("conv", dict(seqlen=1 << 31), 2),
    ("ffn", dict(), 0), ("ffn", dict(rows=1, dim=8, hidden=8, activation=2), 0), ("ffn", dict(x_stride=56), 0),
    ("ffn", dict(rows=0), 1), ("ffn", dict(activation=0), 1), ("ffn", dict(activation=3), 1), ("ffn", dict(io_dtype=7), 1),
    ("ffn", dict(io_dtype=0), 3), ("ffn", dict(dim=44), 2), ("ffn", dict(hidden=100), 2), ("ffn", dict(x_stride=50), 2),
    ("ffn", dict(x_stride=40), 2), ("ffn", dict(rows=(1 << 24) + 1), 2),
])
def test_problem_checks(cuda_lib, kind, over, code):
    assert size_status(cuda_lib, kind, struct(kind, **over)) == code


def test_sizes(cuda_lib):
    for kind in ("glr", "conv", "ffn"):
        assert size_status(cuda_lib, kind, None) == 1
    marks = 2 * 13 * 48 * 4  # every eighth step's states
    assert binding.ssd_glr_stash_size(struct("glr")) == marks
    a, b = (binding.ssd_glr_workspace_size(struct("glr"), s) for s in (False, True))
    assert b < a and a - b >= marks
    assert binding.ssd_glr_stash_size(struct("glr", packed=1)) == marks // 2  # 100 steps in all
    assert binding.ssd_glr_stash_size(struct("glr", io_dtype=0)) == 2 * 25 * 48 * 4  # every fourth in fp32
    assert binding.ssd_ffn_stash_size(struct("ffn")) == 128 * 96 * 6
    p = struct("ffn")
    assert 256 <= binding.ssd_ffn_workspace_size(p, False) < binding.ssd_ffn_workspace_size(p, True, True)
    assert binding.ssd_ffn_workspace_size(p, True) - binding.ssd_ffn_workspace_size(p, True, True) >= 128 * 96 * 6


F = 1 << 20  # never dereferenced


def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("uses fake device addresses; host-only check")


def test_glr_calls_refuse_bad_pointers(cuda_lib):
    no_gpu()
    p, big = struct("glr"), 1 << 40
    fwd = lambda p=p, x=F, r=F, i=F, lam=F, h0=None, cu=None, scale=8.0, y=F, hf=F, stash=None, sb=0: (  # noqa: E731
        cuda_lib.ssd_glr_forward(ctypes.byref(p), x, r, i, lam, h0, cu, scale, y, hf, stash, sb, None))
    for name in ("x", "r", "i", "lam", "y"):
        assert fwd(**{name: None}) == 1, name
    for name in ("x", "r", "i", "cu", "h0", "lam", "hf", "stash"):
        over = dict(p=struct("glr", packed=1), cu=F, sb=big)
        assert fwd(**{**over, name: F + 1}) == 4, name
    assert fwd(y=F + 8) == 4 and fwd(stash=F + 8, sb=big) == 4 and fwd(stash=F, sb=2 * 4 * 48 * 4 - 1) == 5
    assert fwd(cu=F) == 1 and fwd(p=struct("glr", packed=1)) == 1
    for bad in (-1.0, float("nan"), float("inf")):
        assert fwd(scale=bad) == 1
    bwd = lambda p=p, **o: cuda_lib.ssd_glr_backward(  # noqa: E731
        ctypes.byref(p), *(o.get(n, F) for n in ("dy", "dhf", "x", "r", "i", "lam")), None, None, o.get("scale", 8.0),
        *(o.get(n, F) for n in ("dx", "dr", "di", "dlam", "dh0")), o.get("stash"), o.get("sb", 0), o.get("ws", F),
        o.get("nb", big), None)
    for name in ("dy", "x", "r", "i", "lam", "dx", "dr", "di", "dlam", "ws"):
        assert bwd(**{name: None}) == 1, name
    for name in ("dx", "dr", "di", "ws"):
        assert bwd(**{name: F + 8}) == 4, name
    for name in ("dy", "dhf", "dlam", "dh0"):
        assert bwd(**{name: F + 1}) == 4, name
    assert bwd(nb=binding.ssd_glr_workspace_size(p) - 1) == 5 and bwd(stash=F, sb=1) == 5
    step = lambda p=p, x=F, lam=F, state=F, slots=None, n=2, y=F, scale=8.0: cuda_lib.ssd_glr_step(  # noqa: E731
        ctypes.byref(p), x, F, F, lam, state, slots, n, scale, y, None)
    assert step(x=None) == 1 and step(state=None) == 1 and step(y=None) == 1 and step(lam=None) == 1 and step(n=0) == 1
    assert step(n=1) == 1 and step(p=struct("glr", packed=1)) == 1 and step(scale=-1.0) == 1
    assert step(slots=F + 2) == 4 and step(x=F + 1) == 4 and step(state=F + 2) == 4 and step(y=F + 1) == 4


def test_conv_calls_refuse_bad_pointers(cuda_lib):
    no_gpu()
    p, big = struct("conv"), 1 << 40
    fwd = lambda p=p, x=F, w=F, b=None, taps=None, cu=None, y=F, last=None: cuda_lib.ssd_conv_forward(  # noqa: E731
        ctypes.byref(p), x, w, b, taps, cu, y, last, None)
    assert fwd(x=None) == 1 and fwd(w=None) == 1 and fwd(y=None) == 1 and fwd(cu=F) == 1
    assert fwd(p=struct("conv", packed=1)) == 1 and fwd(p=struct("conv", packed=1), cu=F + 2) == 4
    for name in ("x", "y", "taps", "last"):
        assert fwd(**{name: F + 1}) == 4, name
    assert fwd(w=F + 2) == 4 and fwd(b=F + 2) == 4
    bwd = lambda **o: cuda_lib.ssd_conv_backward(  # noqa: E731
        ctypes.byref(p), *(o.get(n, F) for n in ("dy", "x", "w", "b", "taps")), None,
        *(o.get(n, F) for n in ("dx", "dw", "db", "dtaps", "ws")), o.get("nb", big), None)
    for name in ("dy", "x", "w", "dx", "ws"):
        assert bwd(**{name: None}) == 1, name
    for name in ("dy", "x", "dx", "dtaps", "taps", "ws"):
        assert bwd(**{name: F + 1}) == 4, name
    assert bwd(dw=F + 2) == 4 and bwd(nb=binding.ssd_conv_workspace_size(p) - 1) == 5
    step = lambda p=p, x=F, state=F, slots=None, n=2, y=F: cuda_lib.ssd_conv_step(  # noqa: E731
        ctypes.byref(p), x, F, None, state, slots, n, y, None)
    assert step(x=None) == 1 and step(state=None) == 1 and step(y=None) == 1 and step(n=0) == 1 and step(n=1) == 1
    assert step(p=struct("conv", packed=1)) == 1 and step(slots=F + 1) == 4 and step(state=F + 1) == 4


def test_ffn_calls_refuse_bad_pointers(cuda_lib):
    no_gpu()
    p, big = struct("ffn"), 1 << 40
    fwd = lambda **o: cuda_lib.ssd_ffn_forward(ctypes.byref(p), *(o.get(n, F) for n in ("x", "wg", "wu", "h")),  # noqa: E731
                                               o.get("stash"), o.get("sb", 0), o.get("ws", F), o.get("nb", big), None)
    for name in ("x", "wg", "wu", "h", "ws"):
        assert fwd(**{name: None}) == 1 and fwd(**{name: F + 8}) == 4, name
    assert fwd(stash=F + 8, sb=big) == 4 and fwd(stash=F, sb=128 * 96 * 6 - 1) == 5 and fwd(nb=255) == 5
    bwd = lambda **o: cuda_lib.ssd_ffn_backward(  # noqa: E731
        ctypes.byref(p), *(o.get(n, F) for n in ("dh", "x", "wg", "wu", "dx", "dwg", "dwu")), o.get("stash"), o.get("sb", 0),
        o.get("ws", F), o.get("nb", big), None)
    for name in ("dh", "x", "wg", "wu", "dx", "dwg", "dwu", "ws"):
        assert bwd(**{name: None}) == 1 and bwd(**{name: F + 8}) == 4, name
    assert bwd(nb=binding.ssd_ffn_workspace_size(p, True) - 1) == 5 and bwd(stash=F, sb=1) == 5


# ------------------------------------------------------------- the Python calls
@pytest.fixture
def launched(monkeypatch):
    """The Python calls up to the library's, on CPU tensors that pass for the current device's."""
    seen = []
    for name in ("ssd_glr_forward", "ssd_glr_backward", "ssd_glr_step", "ssd_conv_forward", "ssd_conv_backward",
                 "ssd_conv_step", "ssd_ffn_forward", "ssd_ffn_backward"):
        monkeypatch.setattr(binding, name, lambda prob, *a, name=name: seen.append((name, prob)))
    monkeypatch.setattr(binding, "_device", lambda first, *others: 0)
    monkeypatch.setattr(binding, "_stream", lambda *a: 0)
    return seen


def test_what_the_python_calls_pass_on(cuda_lib, launched):
    wide = torch.zeros((3, 7, 100))
    x, r, i = wide[..., :24], wide[..., 30:54], torch.zeros((3, 7, 24))
    lam, h0 = torch.zeros(24), torch.zeros((3, 24))
    stash = binding.glr_stash(x)
    y, last = binding.glr_forward(x, r, i, lam, h0, stash=stash)
    g = binding.glr_backward(y, x, r, i, lam, h0, h0, stash=stash)
    assert y.shape == (3, 7, 24) and last.shape == (3, 24) and g["dx"].is_contiguous() and g["dh0"].shape == (3, 24)
    p = launched[0][1]
    assert (p.io_dtype, p.packed, p.batch, p.seqlen, p.dim, p.x_stride, p.r_stride, p.i_stride) == (0, 0, 3, 7, 24, 100, 100, 0)
    cu = torch.tensor([0, 3, 7], dtype=torch.int32)
    binding.glr_forward(i[0], r[0], i[0], lam, cu_seqlens=cu)
    p = launched[-1][1]
    assert (p.packed, p.batch, p.seqlen, p.r_stride) == (1, 2, 7, 100)
    one = wide[:, :1, :24]  # one step a batch: the batches are the steps
    binding.glr_step(one, one, one, lam, torch.zeros((5, 24)), torch.zeros(3, dtype=torch.int32))
    assert launched[-1][1].x_stride == 700
    w = torch.zeros((24, 4))
    y, taps = binding.conv_forward(x, w, lam, taps=torch.zeros((3, 3, 24)))
    assert taps.shape == (3, 3, 24) and launched[-1][1].x_stride == 100
    g = binding.conv_backward(y, x, w)
    assert g["db"] is None and g["dtaps"] is None and g["dw"].shape == (24, 4)
    b = torch.zeros((4, 5, 24), dtype=torch.bfloat16)
    wg = torch.zeros((40, 24), dtype=torch.bfloat16)
    assert binding.ffn_forward(b, wg, wg).shape == (4, 5, 40)
    p = launched[-1][1]
    assert (p.io_dtype, p.activation, p.rows, p.dim, p.hidden, p.x_stride) == (1, 1, 20, 24, 40, 0)


@pytest.mark.parametrize("again", [False, True])
def test_python_calls_refuse_tensors_that_do_not_fit(cuda_lib, launched, again):
    """Also after a call whose tensors did (a call is found again by its tensors' types, shapes and strides)."""
    z = lambda *s, **o: torch.zeros(s, **o)  # noqa: E731
    x, lam, w = z(2, 7, 24), z(24), z(24, 4)
    xb, wg = z(6, 24, dtype=torch.bfloat16), z(40, 24, dtype=torch.bfloat16)
    cu = torch.tensor([0, 3, 7], dtype=torch.int32)
    if again:
        binding.glr_forward(x, x, x, lam)
        binding.conv_forward(x, w, lam)
        binding.ffn_forward(xb, wg, wg)
    bad = [lambda: binding.glr_forward(x, x.bfloat16(), x, lam), lambda: binding.glr_forward(x, x, x[:1], lam),
           lambda: binding.glr_forward(x, x, x, lam[:23]), lambda: binding.glr_forward(x, x, x, lam.double()),
           lambda: binding.glr_forward(x, x, x, lam, z(1, 24)), lambda: binding.glr_forward(x, x, x, lam, cu_seqlens=cu),
           lambda: binding.glr_forward(x[0], x[0], x[0], lam, cu_seqlens=cu.long()),
           lambda: binding.glr_forward(x[0, 0], x[0, 0], x[0, 0], lam),
           lambda: binding.glr_forward(x.transpose(0, 1), x.transpose(0, 1), x.transpose(0, 1), lam),
           lambda: binding.glr_forward(x.mT.contiguous().mT, x, x, lam), lambda: binding.glr_forward(x.double(), x.double(), x.double(), lam),
           lambda: binding.glr_backward(x[:, :6], x, x, x, lam), lambda: binding.glr_backward(x.mT.contiguous().mT, x, x, x, lam),
           lambda: binding.glr_backward(x, x, x, x, lam, z(2, 23)),
           lambda: binding.glr_step(x, x, x, lam, z(5, 23)), lambda: binding.glr_step(x, x, x, lam, z(5, 24).double()),
           lambda: binding.glr_step(x, x, x, lam, z(5, 24), z(2).long()),
           lambda: binding.conv_forward(x, w[:23]), lambda: binding.conv_forward(x, w.T.contiguous().T),
           lambda: binding.conv_forward(x, w, lam.bfloat16()), lambda: binding.conv_forward(x, w, activation="relu"),
           lambda: binding.conv_forward(x, w, taps=z(2, 4, 24)), lambda: binding.conv_backward(x.bfloat16(), x, w),
           lambda: binding.conv_step(x, w, None, z(5, 4, 24)), lambda: binding.conv_step(x, w, None, z(5, 3, 24), z(3, dtype=torch.int32)),
           lambda: binding.ffn_forward(xb, wg[:, :16], wg[:, :16]), lambda: binding.ffn_forward(xb, wg, wg[:39]),
           lambda: binding.ffn_forward(xb, wg, wg.float()), lambda: binding.ffn_forward(xb.T.contiguous().T, wg, wg),
           lambda: binding.ffn_forward(xb, wg, wg, activation="tanh"), lambda: binding.ffn_backward(xb, xb, wg, wg)]
    n = len(launched)
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was taken")
    assert len(launched) == n


def test_calls_off_the_current_device_launch_nothing(cuda_lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    x, lam, w = torch.zeros((1, 3, 8)), torch.zeros(8), torch.zeros((8, 4))
    xb = torch.zeros((3, 8), dtype=torch.bfloat16)
    for call in (lambda: binding.glr_forward(x, x, x, lam), lambda: binding.glr_backward(x, x, x, x, lam),
                 lambda: binding.glr_step(x, x, x, lam, torch.zeros((1, 8))), lambda: binding.conv_forward(x, w),
                 lambda: binding.conv_backward(x, x, w), lambda: binding.conv_step(x, w, None, torch.zeros((1, 3, 8))),
                 lambda: binding.ffn_forward(xb, xb, xb), lambda: binding.ffn_backward(torch.zeros((3, 3), dtype=xb.dtype), xb, xb, xb)):
        with pytest.raises(ValueError, match="current"):
            call()
