"""GPU parity of layer norm and its backward pass (through the C ABI) with the formulas in float64.

Bounds (max|gpu - ref| / max|ref|), set before the first run: fp32 sums over D or over the rows leave about 1e-6; 2e-5
for fp32 outputs.  bf16 outputs are rounded once: 4e-3 (2 x 2^-9)."""
import numpy as np
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.bfloat16: 4e-3}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(rows, dim, io, wt, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = (rn(rows, dim) * torch.exp(0.5 * rn(dim)) + 0.7).to(TYPES[io])
    return dict(x=x, w=(1 + 0.3 * rn(dim)).to(TYPES[wt]), b=rn(dim).to(TYPES[wt]), dy=rn(rows, dim).to(TYPES[io]))


def reference(c, eps, w=True, b=True):
    x, dy = c["x"].double().numpy(), c["dy"].double().numpy()
    wt = c["w"].double().numpy() if w else np.ones(x.shape[1])
    bt = c["b"].double().numpy() if b else np.zeros(x.shape[1])
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    h = (x - mean) * rstd
    g = dy * wt
    dx = rstd * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dict(y=h * wt + bt, mean=mean[:, 0], rstd=rstd[:, 0], dx=dx, dw=(dy * h).sum(0), db=dy.sum(0))


def check(name, got, ref, scale=None):
    x = got.double().cpu().numpy()
    assert x.shape == ref.shape and np.isfinite(x).all(), name
    top = max(float(np.abs(ref).max()) if scale is None else scale, 1e-30)
    err = float(np.abs(x - ref).max()) / top
    assert err <= TOL[got.dtype], (name, err)


# every width class of the launch rule, both sides of its limits, whole and ragged 16-byte pieces
SIZES = [(1, 1), (3, 2), (5, 7), (33, 64), (40, 128), (17, 129), (9, 256), (20, 257), (6, 512), (7, 513), (31, 1000),
         (5, 1024), (4, 1025), (12, 2048), (700, 2056), (3, 2560), (2, 4096), (2, 4097), (1, 8192), (2, 8193), (3, 16384),
         (1300, 96), (5000, 8)]


@pytest.mark.parametrize("rows,dim", SIZES)
@pytest.mark.parametrize("io,wt", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_matches_float64(rows, dim, io, wt):
    c = make(rows, dim, io, wt, 1)
    eps = 1e-3 if dim < 8 else 1e-5  # a row of two values can lie closer together than fp32 resolves
    ref = reference(c, eps)
    d = {k: t.cuda() for k, t in c.items()}
    y, mean, rstd = binding.norm_forward(d["x"], d["w"], d["b"], eps)
    g = binding.norm_backward(d["dy"], d["x"], mean, rstd, d["w"])
    torch.cuda.synchronize()
    check("y", y, ref["y"])
    check("mean", mean, ref["mean"])
    check("rstd", rstd, ref["rstd"])
    # dx of one or two columns is a difference of equal numbers: its size is that of its terms
    size = float((np.abs(c["dy"].double().numpy() * c["w"].double().numpy()) * ref["rstd"][:, None]).max())
    check("dx", g["dx"], ref["dx"], max(size, float(np.abs(ref["dx"]).max())))
    check("dw", g["dw"], ref["dw"], max(float(np.abs(ref["dw"]).max()), 1e-2))
    check("db", g["db"], ref["db"])


def test_without_weight_bias_or_weight_gradients():
    c = make(50, 300, "bf16", "f32", 2)
    d = {k: t.cuda() for k, t in c.items()}
    for w, b in ((None, None), (d["w"], None), (None, d["b"])):
        ref = reference(c, 1e-5, w is not None, b is not None)
        y, mean, rstd = binding.norm_forward(d["x"], w, b)
        check("y", y, ref["y"])
        g = binding.norm_backward(d["dy"], d["x"], mean, rstd, w)
        for n in ("dx", "dw", "db"):
            check(n, g[n], ref[n])
        prob = binding.norm_problem(d["x"], w)
        dx = torch.empty_like(d["x"])
        binding.ssd_norm_backward(prob, d["dy"], d["x"], mean, rstd, w, dx, None, None, None, 0)
        assert torch.equal(dx, g["dx"])
        y2 = torch.empty_like(y)
        binding.ssd_norm_forward(prob, d["x"], w, b, 1e-5, y2, None, None)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("at,width", [(0, 264), (8, 300), (1, 261)])
def test_rows_of_a_wider_tensor(io, at, width):
    c = make(37, 240, io, "f32", 3)
    d = {k: t.cuda() for k, t in c.items()}
    wide = torch.full((37, width), float("nan"), dtype=TYPES[io], device="cuda")
    wide[:, at:at + 240] = d["x"]
    x = wide[:, at:at + 240]
    y, mean, rstd = binding.norm_forward(x, d["w"], d["b"])
    g = binding.norm_backward(d["dy"], x, mean, rstd, d["w"])
    ref = reference(c, 1e-5)
    for n, t in dict(g, y=y, mean=mean, rstd=rstd).items():
        check(n, t, ref[n])


def test_constant_rows_and_large_offsets():
    """Rows of one value (variance zero) and rows whose mean is a thousand times their width."""
    x = torch.full((4, 512), 3.0)
    x[2:] = 1000 + torch.randn((2, 512), generator=torch.Generator().manual_seed(1))
    c = dict(x=x, w=torch.ones(512), b=torch.zeros(512), dy=torch.ones(4, 512))
    y, mean, rstd = binding.norm_forward(x.cuda(), c["w"].cuda(), c["b"].cuda())
    assert (y[:2] == 0).all()
    ref = reference(c, 1e-5)
    # the mean of numbers near 1000 carries 2^-24 x 1000 of the rows' width of 1
    assert np.abs(y.double().cpu().numpy() - ref["y"]).max() <= 5e-4
    assert np.abs(rstd[2:].double().cpu().numpy() / ref["rstd"][2:] - 1).max() <= 1e-5


def test_rows_take_nothing_from_a_nan_row_and_calls_repeat():
    c = make(300, 320, "bf16", "f32", 4)
    d = {k: t.cuda() for k, t in c.items()}
    y, mean, rstd = binding.norm_forward(d["x"], d["w"], d["b"])
    g, g2 = (binding.norm_backward(d["dy"], d["x"], mean, rstd, d["w"]) for _ in range(2))
    for n in g:
        assert torch.equal(g[n], g2[n]), n
    x = d["x"].clone()
    x[7] = float("nan")
    x[9, 3] = float("inf")
    y2, mean2, rstd2 = binding.norm_forward(x, d["w"], d["b"])
    dx2 = binding.norm_backward(d["dy"], x, mean2, rstd2, d["w"])["dx"]
    keep = [i for i in range(300) if i not in (7, 9)]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(g["dx"][keep], dx2[keep])
    assert y2[7].isnan().all()


def test_offsets_past_32_bits():
    rows, dim = (1 << 31) // 8192 + 5, 8192
    x = torch.zeros((rows, dim), dtype=torch.bfloat16, device="cuda")
    c = make(3, dim, "bf16", "f32", 6)
    d = {k: t.cuda() for k, t in c.items()}
    x[-3:] = d["x"]
    y, mean, rstd = binding.norm_forward(x, d["w"], d["b"])
    ref = reference(c, 1e-5)
    for n, t in dict(y=y, mean=mean, rstd=rstd).items():
        check(n, t[-3:], ref[n])


def test_gradients_against_differences():
    c = make(6, 40, "f32", "f32", 5)
    d = {k: t.cuda() for k, t in c.items()}
    _, mean, rstd = binding.norm_forward(d["x"], d["w"], d["b"])
    g = binding.norm_backward(d["dy"], d["x"], mean, rstd, d["w"])
    f = {k: t.double() for k, t in c.items()}
    for n in ("x", "w", "b"):
        grad = g["d" + n].double().cpu()
        way = grad / grad.norm()
        h = 1e-6
        plus, minus = (float((f["dy"].numpy() * reference({**f, n: f[n] + s * h * way}, 1e-5)["y"]).sum()) for s in (1, -1))
        fd = (plus - minus) / (2 * h)
        assert abs(fd - float(grad.norm())) <= 1e-4 * abs(fd), n


def test_refusals():
    x = torch.randn((4, 32), device="cuda")
    w = torch.ones(32, device="cuda")
    y, mean, rstd = binding.norm_forward(x, w)
    for bad in (lambda: binding.norm_forward(x.half()), lambda: binding.norm_forward(x, w[:16]),
                lambda: binding.norm_forward(x.t()), lambda: binding.norm_forward(x, w, w.bfloat16()),
                lambda: binding.norm_backward(y[:2], x, mean, rstd, w), lambda: binding.norm_backward(y.bfloat16(), x, mean, rstd, w)):
        with pytest.raises(ValueError):
            bad()

    def status(f):
        try:
            f()
        except binding.SSDError as e:
            return e.status
        return 0

    prob = binding.norm_problem(x, w)
    fwd = lambda p=prob, xx=x, yy=y, eps=1e-5: status(  # noqa: E731
        lambda: binding.ssd_norm_forward(p, xx, w, None, eps, yy, mean, rstd))
    assert fwd() == 0 and fwd(xx=None) == 1 and fwd(yy=None) == 1 and fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1
    assert fwd(xx=x.data_ptr() + 2) == 4 and fwd(yy=y.data_ptr() + 8) == 4
    big = binding.norm_problem(x, w)
    big.dim = 16385
    assert fwd(p=big) == 2
    big.dim, big.x_stride = 32, 31
    assert fwd(p=big) == 2
    big.x_stride, big.rows = 0, 0
    assert fwd(p=big) == 1
    big.rows, big.io_dtype = 4, 9
    assert fwd(p=big) == 1
    n = binding.ssd_norm_workspace_size(prob)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    bwd = lambda dwp=dw, wsp=ws, nb=n: status(  # noqa: E731
        lambda: binding.ssd_norm_backward(prob, y, x, mean, rstd, w, dx, dwp, None, wsp, nb))
    assert bwd() == 0 and bwd(nb=n - 1) == 5 and bwd(wsp=None) == 1 and bwd(dwp=None, wsp=None, nb=0) == 0
    torch.cuda.synchronize()
