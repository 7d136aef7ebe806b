"""Workloads of the gated delta rule (one decay per head) and of layer norm.

Five operators, by the calls a program makes:

* ``prefill``  the chunked delta rule over whole prompts, equal or packed (o and the final state);
* ``train``    its forward and backward pass (o and the gradients of q, k, v, g, beta);
* ``step``     its form for one or a few tokens per sequence, on a cache of states updated in place;
* ``norm``     layer norm's forward pass (y, mean, rstd);
* ``normtrain`` layer norm's forward and backward pass, with the reductions of the weight's and the bias's gradient.

Per sequence and value head, with state S [K, V], one step of the delta rule is

    S <- exp(g) S;   r = beta (v - S^T k);   S <- S + k r^T;   o = scale S^T q

``run`` computes the same thing in elementary torch operations in 32 bits (``own`` false) or by the library's calls
(``own`` true); ``exact`` walks the definition step by step in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64  # tokens that the plain form takes at a time
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    d = dict(K=128, V=128, H=8, HV=16)
    return [
        # a chat turn's few words on a small model: latency counts
        dict(name="prefill_short", op="prefill", N=1, T=37, K=64, V=64, H=2, HV=4, packed=False, s0=False, gates="bf16"),
        # one long document: few chains, each of them long
        dict(name="prefill_long", op="prefill", N=1, T=16384, packed=False, s0=False, gates="f32", **d),
        # a server's batch of prompts of many lengths, each continued from a state it has; head widths that end inside
        # a tile
        dict(name="prefill_packed", op="prefill", N=24, T=20011, K=128, V=96, H=16, HV=32, packed=True, s0=True,
             gates="f32"),
        # the repository's delta-rule workload (b 2, T 1024, 8 / 16 heads of 128), in bf16
        dict(name="train_base", op="train", N=2, T=1024, **d),
        # a layer of a large model at a full batch: the longest call
        dict(name="train_large", op="train", N=4, T=4096, K=128, V=128, H=16, HV=32),
        # one user, one token
        dict(name="step_one", op="step", N=1, T=1, slots=1, io="bf16", **d),
        # a full serving batch, one token each, states in a cache of slots
        dict(name="step_batch", op="step", N=192, T=1, K=128, V=128, H=16, HV=32, slots=256, io="bf16"),
        # a few drafted tokens for each of a batch, in fp32
        dict(name="step_draft", op="step", N=16, T=5, slots=16, io="f32", **d),
        # one token's norm in front of a mixer
        dict(name="norm_token", op="norm", rows=1, dim=2560, io="bf16", weights="f32"),
        # the norm of each head's output, over a prompt: many short rows
        dict(name="norm_heads", op="norm", rows=16384 * 16, dim=128, io="bf16", weights="f32"),
        # the norm in front of the mixer in a training step (2.7B layer shape: 4 x 4096 tokens, width 2560)
        dict(name="normtrain_large", op="normtrain", rows=16384, dim=2560, io="bf16", weights="f32"),
        # an odd width and an odd number of rows, in fp32
        dict(name="normtrain_odd", op="normtrain", rows=1501, dim=1537, io="f32", weights="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "step", "norm", "normtrain"])
    if op in ("norm", "normtrain"):
        dim = _log(rng, 64, 8192)
        rows = _log(rng, 1, max(1, min(1 << 18, 40_000_000 // dim)))
        return dict(op=op, rows=rows, dim=dim, io=rng.choice(["bf16", "f32"]), weights=rng.choice(["bf16", "f32"]))
    H = rng.choice([1, 2, 3, 4, 8, 16])
    HV = H * rng.choice([1, 2, 2, 4])
    K, V = rng.choice([(64, 64), (128, 128), (128, 128), (128, 64), (96, 128), (72, 40), (128, 100)])
    c = dict(op=op, H=H, HV=HV, K=K, V=V)
    if op == "step":
        N = _log(rng, 1, max(1, min(256, 6144 // HV)))
        return dict(c, N=N, T=rng.choice([1, 1, 1, 2, 3, 7]), slots=N + rng.randrange(0, 9),
                    io=rng.choice(["bf16", "f32"]))
    most = (4 * 4096 * 32 if op == "train" else 16384 * 32) // HV
    N = _log(rng, 1, 16)
    T = _log(rng, 1 if op == "prefill" else 16, min(8192, most // N))
    if op == "train":
        return dict(c, N=N, T=T)
    packed = rng.random() < 0.5
    return dict(c, N=N, T=max(T * N, N) if packed else T, packed=packed, s0=rng.random() < 0.5,
                gates=rng.choice(["bf16", "f32"]))


def _lengths(case, seed):
    """Lengths of a packed batch: spread over a factor of about ten, some of a few tokens; their sum is T."""
    n, t = case["N"], case["T"]
    g = torch.Generator().manual_seed(seed ^ 0x5EED)
    w = torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * 2.3)
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * t).long()
    cut[-1] = t
    return [int(b - a) for a, b in zip([0] + cut[:-1].tolist(), cut.tolist())]


# ------------------------------------------------------------------------------------------------ their inputs
def _gates(shape, gen, dtype):
    """g and beta as a mixer makes them: g = -A softplus(a + bias) with A in 1..16 a head and time steps of 1e-3 to 0.1
    (so a step keeps from nearly all to a fifth of the state), beta = sigmoid(b)."""
    hv = shape[-1]
    dev = gen.device
    a = 1.0 + 15.0 * torch.rand(hv, generator=gen, device=dev)
    dt = torch.exp(torch.rand(hv, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))
    bias = dt + torch.log(-torch.expm1(-dt))
    g = -a * torch.nn.functional.softplus(torch.randn(shape, generator=gen, device=dev) + bias)
    beta = torch.sigmoid(torch.randn(shape, generator=gen, device=dev))
    return g.to(dtype), beta.to(dtype)


def _keys(shape, gen, dtype):
    """Queries and keys as a mixer makes them: unit length, after an activation that leaves them mostly positive, so
    that neighbouring keys are far from orthogonal."""
    x = torch.nn.functional.silu(torch.randn(shape, generator=gen, device=gen.device) + 0.3)
    return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("norm", "normtrain"):
        io, wt = TYPES[case["io"]], TYPES[case["weights"]]
        rows, dim = case["rows"], case["dim"]
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        # a residual stream: columns of their own offsets and widths, rows of their own size
        x = randn(rows, dim) * torch.exp(0.5 * randn(dim)) + 0.3 * randn(dim) + 0.5
        s = dict(case=case, x=(x * torch.exp(0.3 * randn(rows, 1))).to(io), w=(1 + 0.2 * randn(dim)).to(wt),
                 b=(0.1 * randn(dim)).to(wt))
        if op == "normtrain":
            s["dy"] = randn(rows, dim).to(io)
        return s
    n, t, h, hv, k, v = (case[x] for x in ("N", "T", "H", "HV", "K", "V"))
    packed = case.get("packed", False)
    lead = (1, t) if packed else (n, t)
    io = TYPES[case.get("io", "bf16")]
    s = dict(case=case, q=_keys(lead + (h, k), gen, io), k=_keys(lead + (h, k), gen, io),
             v=torch.randn(lead + (hv, v), generator=gen, device="cuda").to(io), scale=k ** -0.5)
    s["g"], s["beta"] = _gates(lead + (hv,), gen, TYPES[case.get("gates", "bf16")])
    s["cfg"] = dict(dtype=case.get("io", "bf16"), gate_dtype=case.get("gates", "bf16"), batch=n, seqlen=t, nheads=h,
                    value_heads=hv, key_dim=k, value_dim=v)
    if packed:
        s["lengths"] = _lengths(case, seed)
        cu = torch.cumsum(torch.tensor([0] + s["lengths"]), 0)
        s["cu"] = cu.to(device="cuda", dtype=torch.int32)
    if case.get("s0"):
        s["s0"] = 0.1 * torch.randn((n, hv, k, v), generator=gen, device="cuda")
    if op == "train":
        s["do"] = torch.randn(lead + (hv, v), generator=gen, device="cuda").to(io)
    if op == "step":
        s["state"] = 0.1 * torch.randn((case["slots"], hv, k, v), generator=gen, device="cuda")
        s["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
    return s


# ------------------------------------------------------------------------------------------------ the plain forms
def _unit_lower_inverse(a):
    """(I + a)^-1 for strictly lower triangular a [.., C, C], C a power of two: blocks of twice the size at a time."""
    c = a.shape[-1]
    i = torch.arange(c, device=a.device)
    inv = torch.eye(c, device=a.device, dtype=a.dtype).expand_as(a)
    size = 1
    while size < c:
        off = (i[:, None] // (2 * size) == i // (2 * size)) & (i[:, None] // size != i // size)
        inv = inv - inv @ (a * off) @ inv
        size *= 2
    return inv


def _plain_delta(q, k, v, g, beta, s0, scale):
    """The delta rule by chunks, fp32: q, k [N, T, H, K], v [N, T, HV, V], g, beta [N, T, HV]; o [N, T, HV, V] and the
    final state [N, HV, K, V]."""
    n, t, h, kd = q.shape
    hv, vd = v.shape[2:]
    nc = -(-t // CHUNK)

    def chunks(x, heads):  # [N, T, heads(, D)] -> [N, HV, nc, C(, D)]; missing steps are zeros, which change nothing
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, nc * CHUNK - t))
        x = x.unflatten(1, (nc, CHUNK)).movedim(3, 1)
        return x.repeat_interleave(hv // heads, dim=1) if heads != hv else x

    q, k, v, g, beta = chunks(q, h), chunks(k, h), chunks(v, hv), chunks(g, hv), chunks(beta, hv)
    cum = torch.cumsum(g, -1)
    i = torch.arange(CHUNK, device=q.device)
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(i[:, None] < i, -math.inf))
    a = beta[..., None] * decay * (k @ k.mT) * (i[:, None] > i)
    inv = _unit_lower_inverse(a)
    u = inv @ (beta[..., None] * v)
    w = inv @ ((beta * torch.exp(cum))[..., None] * k)
    p = scale * decay * (q @ k.mT)
    qe = scale * torch.exp(cum)[..., None] * q
    ke = torch.exp(cum[..., -1:] - cum)[..., None] * k
    keep = torch.exp(cum[..., -1])[..., None, None]
    s = torch.zeros((n, hv, kd, vd), device=q.device) if s0 is None else s0
    out = []
    for c in range(nc):  # the state passes from chunk to chunk
        r = u[:, :, c] - w[:, :, c] @ s
        out.append(qe[:, :, c] @ s + p[:, :, c] @ r)
        s = keep[:, :, c] * s + ke[:, :, c].mT @ r
    o = torch.stack(out, 2).movedim(1, 3).flatten(1, 2)[:, :t]
    return o, s


def _plain_prefill(s):
    x = [s[n].float() for n in ("q", "k", "v", "g", "beta")]
    if "lengths" not in s:
        o, final = _plain_delta(*x, s.get("s0"), s["scale"])
        return o.to(s["v"].dtype), final
    at = torch.arange(s["case"]["T"], device="cuda")
    cu = s["cu"].long()
    row = torch.searchsorted(cu, at, right=True) - 1
    col = at - cu[row]
    wide = [y.new_zeros((s["case"]["N"], max(s["lengths"])) + y.shape[2:]) for y in x]
    for y, z in zip(x, wide):
        z[row, col] = y[0]
    o, final = _plain_delta(*wide, s.get("s0"), s["scale"])
    return o[row, col][None].to(s["v"].dtype), final


def _plain_train(s):
    with torch.enable_grad():
        x = [s[n].float().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
        o, _ = _plain_delta(*x, None, s["scale"])
        grads = torch.autograd.grad(o, x, s["do"].float())
    o = o.detach().to(s["v"].dtype)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta"), (y.to(s[n].dtype) for y, n in zip(grads, ("q", "k", "v", "g", "beta")))),
                o=o)


def _plain_step(s):
    group = s["case"]["HV"] // s["case"]["H"]
    q, k = (s[n].float().repeat_interleave(group, 2) for n in ("q", "k"))
    v, g, beta = (s[n].float() for n in ("v", "g", "beta"))
    at = s["slots"].long()
    state = s["state"][at]
    out = []
    for t in range(s["case"]["T"]):
        state = torch.exp(g[:, t])[..., None, None] * state
        r = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * state).sum(-2))
        state = state + k[:, t, :, :, None] * r[:, :, None, :]
        out.append(s["scale"] * (q[:, t, :, :, None] * state).sum(-2))
    s["state"][at] = state
    return torch.stack(out, 1).to(s["v"].dtype), s["state"]


def _plain_norm(s):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    xh = xc * rstd
    y = (xh * w + b).to(s["x"].dtype)
    if "dy" not in s:
        return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0])
    dy = s["dy"].float()
    wdy = dy * w
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
    return dict(y=y, dx=dx.to(s["x"].dtype), dw=(dy * xh).sum(0).to(s["w"].dtype), db=dy.sum(0).to(s["b"].dtype))


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"prefill": _plain_prefill, "train": _plain_train, "step": _plain_step, "norm": _plain_norm,
                "normtrain": _plain_norm}[op](s)
    from selective_state_space_ssd_gb300 import binding

    if op == "prefill":
        return binding.delta_forward(s["cfg"], s["q"], s["k"], s["v"], s["g"], s["beta"], s.get("s0"), s["scale"],
                                     cu_seqlens=s.get("cu"))
    if op == "train":
        x = (s["q"], s["k"], s["v"], s["g"], s["beta"])
        stash = binding.delta_stash(s["cfg"], s["q"].device)
        o, _ = binding.delta_forward(s["cfg"], *x, scale=s["scale"], stash=stash)
        grads = binding.delta_backward(s["cfg"], s["do"], *x, scale=s["scale"], stash=stash)
        return dict({n: grads[n] for n in ("dq", "dk", "dv", "dg", "dbeta")}, o=o)
    if op == "step":
        o = binding.delta_step(s["cfg"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slots"], s["scale"])
        return o, s["state"]
    y, mean, rstd = binding.norm_forward(s["x"], s["w"], s["b"], EPS)
    if op == "norm":
        return dict(y=y, mean=mean, rstd=rstd)
    grads = binding.norm_backward(s["dy"], s["x"], mean, rstd, s["w"])
    return dict(y=y, dx=grads["dx"], dw=grads["dw"], db=grads["db"])


# ------------------------------------------------------------------------------------------------ the definition, 64 bits
def _walk(q, k, v, g, beta, s, scale):
    """Step by step: q, k [T, .., K], v [T, .., V], g, beta [T, ..], s [.., K, V]; o [T, .., V] and the last state."""
    o = torch.empty_like(v)
    for t in range(q.shape[0]):
        s = torch.exp(g[t])[..., None, None] * s
        r = beta[t][..., None] * (v[t] - (k[t][..., None, :] @ s)[..., 0, :])
        s = s + k[t][..., :, None] * r[..., None, :]
        o[t] = scale * (q[t][..., None, :] @ s)[..., 0, :]
    return o, s


def _walk_back(q, k, v, g, beta, scale, do):
    """The reverse walk of <do, o> from an empty first state; states are kept for 64 steps at a time."""
    steps = q.shape[0]
    s = q.new_zeros(k.shape[1:] + (v.shape[-1],))
    marks, o = [], []
    for a in range(0, steps, 64):
        marks.append(s)
        part, s = _walk(*(x[a:a + 64] for x in (q, k, v, g, beta)), s, scale)
        o.append(part)
    dq, dk, dv, dg, dbeta = (torch.empty_like(x) for x in (q, k, v, g, beta))
    ds = torch.zeros_like(s)
    for m in reversed(range(len(marks))):
        a, b = 64 * m, min(steps, 64 * m + 64)
        before = [marks[m]]
        for t in range(a, b):
            before.append(_walk(*(x[t:t + 1] for x in (q, k, v, g, beta)), before[-1], scale)[1])
        for t in reversed(range(a, b)):
            faded = torch.exp(g[t])[..., None, None] * before[t - a]
            miss = v[t] - (k[t][..., None, :] @ faded)[..., 0, :]
            ds = ds + scale * q[t][..., :, None] * do[t][..., None, :]
            dq[t] = scale * (before[t - a + 1] @ do[t][..., None])[..., 0]
            dr = (k[t][..., None, :] @ ds)[..., 0, :]
            dv[t] = beta[t][..., None] * dr
            dbeta[t] = (dr * miss).sum(-1)
            dk[t] = (ds @ (beta[t][..., None] * miss)[..., None])[..., 0] - (faded @ dv[t][..., None])[..., 0]
            ds = ds - k[t][..., :, None] * dv[t][..., None, :]
            dg[t] = (ds * faded).sum((-1, -2))
            ds = torch.exp(g[t])[..., None, None] * ds
    return torch.cat(o), dq, dk, dv, dg, dbeta


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "normtrain"):
        with torch.enable_grad():
            x, w, b = (s[n].double().requires_grad_() for n in ("x", "w", "b"))
            mean = x.sum(1) / case["dim"]
            var = ((x - mean[:, None]) ** 2).sum(1) / case["dim"]
            y = (x - mean[:, None]) / torch.sqrt(var[:, None] + EPS) * w + b
            if op == "norm":
                return dict(y=y.detach(), mean=mean.detach(), rstd=(var.detach() + EPS) ** -0.5)
            dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].double())
        return dict(y=y.detach(), dx=dx, dw=dw, db=db)
    group = case["HV"] // case["H"]
    q, k = (s[n].double().repeat_interleave(group, 2).movedim(1, 0) for n in ("q", "k"))
    v, g, beta = (s[n].double().movedim(1, 0) for n in ("v", "g", "beta"))
    if op == "train":
        o, dq, dk, dv, dg, dbeta = (x.movedim(0, 1) for x in _walk_back(q, k, v, g, beta, s["scale"], s["do"].double().movedim(1, 0)))
        dq, dk = (x.unflatten(2, (case["H"], group)).sum(3) for x in (dq, dk))
        return dict(o=o, dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta)
    if op == "step":
        at = s["slots"].long()
        o, last = _walk(q, k, v, g, beta, s["state"][at].double(), s["scale"])
        full = s["state"].double()
        full[at] = last
        return o.movedim(0, 1), full
    s0 = s["s0"].double() if "s0" in s else v.new_zeros((case["N"], case["HV"], case["K"], case["V"]))
    if "lengths" not in s:
        o, last = _walk(q, k, v, g, beta, s0, s["scale"])
        return o.movedim(0, 1), last
    a, outs, lasts = 0, [], []
    for n, length in enumerate(s["lengths"]):
        o, last = _walk(*(x[a:a + length, 0] for x in (q, k, v, g, beta)), s0[n], s["scale"])
        outs.append(o)
        lasts.append(last)
        a += length
    return torch.cat(outs)[None], torch.stack(lasts)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm", "normtrain"):
        e, w, n = (4 if case["io"] == "f32" else 2), (4 if case["weights"] == "f32" else 2), case["rows"] * case["dim"]
        if op == "norm":
            return dict(bytes=2 * n * e + 2 * case["dim"] * w + 8 * case["rows"], flops=8 * n)
        return dict(bytes=4 * n * e + 4 * case["dim"] * w, flops=20 * n)
    n, t, h, hv, k, v = (case[x] for x in ("N", "T", "H", "HV", "K", "V"))
    tokens = t if case.get("packed") else n * t
    e = 4 if case.get("io") == "f32" else 2
    ge = 4 if case.get("gates") == "f32" else 2
    inputs = tokens * (2 * h * k * e + hv * v * e + 2 * hv * ge)
    o, state = tokens * hv * v * e, n * hv * k * v * 4
    # a step decays the state and reads it with k, writes it with k and reads it with q: 7 K V operations; its
    # backward makes the states again (5) and reads or writes state and gradient nine times more (20)
    if op == "prefill":
        return dict(bytes=inputs + o + state * (2 if case["s0"] else 1), flops=7 * k * v * tokens * hv)
    if op == "train":
        return dict(bytes=2 * inputs + 2 * o, flops=27 * k * v * tokens * hv)
    return dict(bytes=inputs + o + 2 * state + 4 * n, flops=7 * k * v * tokens * hv)
