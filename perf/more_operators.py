"""Workloads of a recurrent block's operators: the gated linear recurrence with one decay per channel, the causal short
convolution in front of it, and the gated feed-forward that follows the mixer.

By the calls a program makes:

* ``scan``       the recurrence over whole prompts, equal or packed (y and the final state);
* ``scantrain``  its forward and backward pass (y and the gradients of x, r, i, lam and the first state);
* ``scanstep``   its form for one or a few tokens per sequence, on a cache of states updated in place;
* ``conv``       the convolution over whole prompts (y and the last inputs of each sequence);
* ``convtrain``  its forward and backward pass (y and the gradients of x, weight and bias);
* ``convstep``   its form for one or a few tokens per sequence, on a cache of inputs updated in place;
* ``ffn``        act(x Wg^T) (x Wu^T);
* ``ffntrain``   its forward and backward pass (h and the gradients of x, Wg and Wu).

Per channel, with sigmoid s and c = 8, a step of the recurrence is

    g = -c softplus(lam) s(r);   a = exp(g);   h <- a h + sqrt(1 - a^2) s(i) x;   y = h

and of the convolution of K taps, weight [D, K] with the present step's tap last,

    z = bias + sum over j < K of weight[:, K - 1 - j] x_{t - j};   y = z s(z)

``run`` computes the same things in elementary torch operations in 32 bits (``own`` false) or by the library's calls
(``own`` true); ``exact`` goes by the definitions in 64 bits.
"""
import math

import torch

own = False

C = 8.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a chat turn's few words on a small model: latency counts
        dict(name="scan_short", op="scan", N=1, T=19, D=1536, packed=False, h0=False, io="bf16"),
        # a server's batch of prompts of many lengths, each continued from a state it has
        dict(name="scan_packed", op="scan", N=24, T=20011, D=2560, packed=True, h0=True, io="bf16"),
        # one long document in a training step: few channels, each of them long
        dict(name="scantrain_long", op="scantrain", N=1, T=16384, D=2560, packed=False, h0=False, io="bf16"),
        # an odd width and an odd length, in fp32
        dict(name="scantrain_odd", op="scantrain", N=3, T=1021, D=1537, packed=False, h0=True, io="f32"),
        # a full serving batch, one token each, states in a cache of slots
        dict(name="scanstep_batch", op="scanstep", N=192, T=1, D=5120, slots=256, io="bf16"),
        # the convolution of the same batch of prompts
        dict(name="conv_packed", op="conv", N=24, T=20011, D=2560, K=4, packed=True, taps=True, io="bf16", weights="f32"),
        # a layer of a large model at a full batch (2.7B layer shape: 4 x 4096 tokens, inner width 5120)
        dict(name="convtrain_large", op="convtrain", N=4, T=4096, D=5120, K=4, io="bf16", weights="f32"),
        # one user, one token
        dict(name="convstep_one", op="convstep", N=1, T=1, D=5120, K=4, slots=1, io="bf16", weights="bf16"),
        # one user, one token: the weights have to be read
        dict(name="ffn_token", op="ffn", M=1, D=2560, F=7680, act="silu"),
        # a serving batch, one token each
        dict(name="ffn_batch", op="ffn", M=192, D=2560, F=7680, act="silu"),
        # ragged sizes on a small model's training step
        dict(name="ffntrain_odd", op="ffntrain", M=1501, D=776, F=2056, act="gelu"),
        # a training step of a layer of a large model: the longest call
        dict(name="ffntrain_large", op="ffntrain", M=8192, D=2560, F=7680, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scantrain", "scantrain", "scanstep", "conv", "convtrain", "convstep", "ffn", "ffn",
                     "ffntrain", "ffntrain"])
    if op in ("ffn", "ffntrain"):
        d, f = 8 * _log(rng, 32, 512), 8 * _log(rng, 64, 1536)
        most = 8192 * 2560 * 7680 // (d * f)
        m = _log(rng, 1 if op == "ffn" else 64, min(16384, max(most, 64)))
        return dict(op=op, M=m, D=d, F=f, act=rng.choice(["silu", "gelu"]))
    d = _log(rng, 64, 6144)
    if rng.random() < 0.7:
        d = max(64, d // 64 * 64)
    io = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, D=d, io=io)
    if op.startswith("conv"):
        c.update(K=rng.choice([4, 4, 4, 3, 2]), weights=rng.choice(["f32", "bf16"]))
    if op in ("scanstep", "convstep"):
        n = _log(rng, 1, 256)
        return dict(c, N=n, T=rng.choice([1, 1, 1, 2, 3, 7]), slots=n + rng.randrange(0, 9))
    n = _log(rng, 1, 32)
    most = 4096 * 10240 // d
    t = _log(rng, 1 if op in ("scan", "conv") else 16, max(16, min(16384 if n == 1 else 4096, most // n)))
    if op == "convtrain":
        return dict(c, N=n, T=t)
    packed = rng.random() < 0.5
    c.update(N=n, T=t * n if packed else t, packed=packed)
    c["taps" if op == "conv" else "h0"] = rng.random() < 0.5
    return c


def _lengths(case, seed):
    """Lengths of a packed batch: spread over a factor of about ten, some of a few tokens; their sum is T."""
    n, t = case["N"], case["T"]
    g = torch.Generator().manual_seed(seed ^ 0x5EED)
    w = torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * 2.3)
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * t).long()
    cut[-1] = t
    return [int(b - a) for a, b in zip([0] + cut[:-1].tolist(), cut.tolist())]


# ------------------------------------------------------------------------------------------------ their inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    op, d = case["op"], case["D"]
    s = dict(case=case)
    if op in ("ffn", "ffntrain"):
        m, f = case["M"], case["F"]
        s["x"] = randn(m, d).to(torch.bfloat16)  # the output of a norm
        s["wg"] = (randn(f, d) * d ** -0.5).to(torch.bfloat16)
        s["wu"] = (randn(f, d) * d ** -0.5).to(torch.bfloat16)
        if op == "ffntrain":
            s["dh"] = randn(m, f).to(torch.bfloat16)
        return s
    n, t, io = case["N"], case["T"], TYPES[case["io"]]
    lead = (t,) if case.get("packed") else (n, t)
    if case.get("packed"):
        s["lengths"] = _lengths(case, seed)
        s["cu"] = torch.cumsum(torch.tensor([0] + s["lengths"]), 0).to(device="cuda", dtype=torch.int32)
    if op.startswith("scan"):
        s["x"] = randn(*lead, d).to(io)
        # both gates come out of one projection: each is a slice of wider rows
        gates = randn(*lead, 2 * d).to(io)
        s["r"], s["i"] = gates[..., :d], gates[..., d:]
        # decays of 0.9 to 0.999 a step where the gate is open
        a = 0.9 + 0.099 * torch.rand(d, generator=gen, device="cuda")
        s["lam"] = torch.log(torch.expm1(-torch.log(a) / C))
        if case.get("h0"):
            s["h0"] = 0.5 * randn(n, d)
        if op == "scantrain":
            s["dy"] = randn(*lead, d).to(io)
        if op == "scanstep":
            s["state"] = 0.5 * randn(case["slots"], d)
    else:
        # the convolved half of a projection whose other half gates the block's output
        s["x"] = randn(*lead, 2 * d).to(io)[..., :d]
        wt, k = TYPES[case["weights"]], case["K"]
        s["w"], s["b"] = (randn(d, k) * k ** -0.5).to(wt), (0.1 * randn(d)).to(wt)
        if case.get("taps"):
            s["taps"] = randn(n, k - 1, d).to(io)
        if op == "convtrain":
            s["dy"] = randn(*lead, d).to(io)
        if op == "convstep":
            s["state"] = randn(case["slots"], k - 1, d).to(io)
    if op.endswith("step"):
        s["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
    return s


# ------------------------------------------------------------------------------------------------ the plain forms
def _rows(s):
    """Of each step of a batch: its sequence and its place in it, [T] for a packed batch, [N, T] for an equal one."""
    n, t = s["case"]["N"], s["case"]["T"]
    at = torch.arange(t, device="cuda")
    if "lengths" not in s:
        return torch.arange(n, device="cuda")[:, None].expand(n, t), at[None].expand(n, t)
    cu = s["cu"].long()
    row = torch.searchsorted(cu, at, right=True) - 1
    return row, at - cu[row]


def _ends(s):
    """The index of each sequence's last step, with those that have one."""
    cu = s["cu"].long()
    return (cu[1:] - 1).clamp_min(0), cu[1:] > cu[:-1]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension -2, twice the span at a time."""
    span = 1
    while span < a.shape[-2]:
        b = torch.cat([b[..., :span, :], b[..., span:, :] + a[..., span:, :] * b[..., :-span, :]], -2)
        a = torch.cat([a[..., :span, :], a[..., span:, :] * a[..., :-span, :]], -2)
        span *= 2
    return b


def _gates(r, i, lam):
    r, i = torch.sigmoid(r), torch.sigmoid(i)
    soft = torch.log1p(torch.exp(lam))
    g = -C * soft * r
    return r, i, soft, g, torch.exp(g), torch.sqrt(-torch.expm1(2 * g))


def _plain_scan(s):
    case, io = s["case"], s["x"].dtype
    x, lam = s["x"].float(), s["lam"]
    r, i, soft, g, a, m = _gates(s["r"].float(), s["i"].float(), lam)
    row, col = _rows(s)
    first = (col == 0)[..., None]
    u = i * x
    start = torch.where(first, s["h0"][row], 0.0) if "h0" in s else torch.zeros_like(x)
    step = torch.where(first, 0.0, a)
    h = _scan(step, m * u + a * start)
    if "lengths" in s:
        end, some = _ends(s)
        none = s["h0"] if "h0" in s else torch.zeros((), device="cuda")
        final = torch.where(some[:, None], h[end], none)
    else:
        final = h[:, -1]
    if case["op"] == "scan":
        return dict(y=h.to(io), h_final=final)
    nxt = torch.cat([step[..., 1:, :], torch.zeros_like(step[..., :1, :])], -2)
    dh = _scan(nxt.flip(-2), s["dy"].float().flip(-2)).flip(-2)
    before = torch.where(first, start, torch.cat([torch.zeros_like(h[..., :1, :]), h[..., :-1, :]], -2))
    q = dh * g * (a * before - a * a / m * u)
    out = dict(y=h.to(io), dx=(dh * m * i).to(io), dr=(q * (1 - r)).to(io), di=(dh * m * u * (1 - i)).to(io),
               dlam=(q.flatten(0, -2).sum(0) * torch.sigmoid(lam) / soft))
    if "h0" in s:
        dh0 = torch.zeros_like(s["h0"])
        where = first[..., 0]
        dh0[row[where]] = (a * dh)[where]
        out["dh0"] = dh0
    return out


def _plain_scanstep(s):
    at = s["slots"].long()
    h = s["state"][at]
    _, i, _, _, a, m = _gates(s["r"].float(), s["i"].float(), s["lam"])
    b = m * i * s["x"].float()
    out = []
    for t in range(s["case"]["T"]):
        h = a[:, t] * h + b[:, t]
        out.append(h)
    s["state"][at] = h
    return dict(y=torch.stack(out, 1).to(s["x"].dtype), state=s["state"])


def _plain_conv(s):
    case, io, wt = s["case"], s["x"].dtype, s["w"].dtype
    k, t = case["K"], case["T"]
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    row, col = _rows(s)

    def back(j):  # the inputs j steps before
        y = torch.cat([torch.zeros_like(x[..., :j, :]), x[..., :t - j, :]], -2) if j < t else torch.zeros_like(x)
        early = (col < j)[..., None]
        if "taps" in s:
            return torch.where(early, s["taps"].float()[row, (k - 1 + col - j).clamp(0, k - 2)], y)
        return torch.where(early, 0.0, y)

    shifted = [back(j) for j in range(k)]
    z = b.expand_as(x)
    for j in range(k):
        z = z + w[:, k - 1 - j] * shifted[j]
    sig = torch.sigmoid(z)
    y = (z * sig).to(io)
    if case["op"] == "conv":
        n = case["N"]
        length = torch.tensor(s["lengths"], device="cuda") if "lengths" in s else torch.full((n,), t, device="cuda")
        begin = s["cu"][:-1].long() if "lengths" in s else torch.arange(n, device="cuda") * t
        flat = s["x"].flatten(0, -2)
        last = torch.zeros((n, k - 1, case["D"]), dtype=io, device="cuda")
        for j in range(k - 1):
            at = length - (k - 1) + j  # this place's step; before the first one, a place of the taps it began with
            old = s["taps"][torch.arange(n, device="cuda"), (at + k - 1).clamp(0, k - 2)] if "taps" in s else 0.0 * last[:, 0]
            new = flat[(begin + at).clamp(0, flat.shape[0] - 1)]
            last[:, j] = torch.where((at >= 0)[:, None], new, old)
        return dict(y=y, taps=last)
    dz = s["dy"].float() * sig * (1 + z * (1 - sig))
    dx = torch.zeros_like(x)
    for j in range(k):
        if j < t:
            dx[..., :t - j, :] += w[:, k - 1 - j] * dz[..., j:, :]
    dw = torch.stack([(dz * shifted[k - 1 - j]).flatten(0, -2).sum(0) for j in range(k)], 1)
    return dict(y=y, dx=dx.to(io), dw=dw.to(wt), db=dz.flatten(0, -2).sum(0).to(wt))


def _plain_convstep(s):
    at, k = s["slots"].long(), s["case"]["K"]
    w, b = s["w"].float(), s["b"].float()
    held = torch.cat([s["state"][at], s["x"]], 1)
    wide = held.float()
    out = []
    for t in range(s["case"]["T"]):
        z = b + (w.T * wide[:, t:t + k]).sum(1)
        out.append(z * torch.sigmoid(z))
    s["state"][at] = held[:, -(k - 1):]
    return dict(y=torch.stack(out, 1).to(s["x"].dtype), state=s["state"])


def _plain_ffn(s):
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.T, x @ wu.T
    if s["case"]["act"] == "silu":
        sig = torch.sigmoid(g)
        act, slope = g * sig, sig * (1 + g * (1 - sig))
    else:
        root = math.sqrt(2 / math.pi)
        th = torch.tanh(root * (g + 0.044715 * g ** 3))
        act, slope = 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * root * (1 + 3 * 0.044715 * g * g)
    h = (act * u).to(s["x"].dtype)
    if "dh" not in s:
        return dict(h=h)
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * act
    return dict(h=h, dx=(dg @ wg + du @ wu).to(s["x"].dtype), dwg=(dg.T @ x).to(s["wg"].dtype),
                dwu=(du.T @ x).to(s["wu"].dtype))


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"scan": _plain_scan, "scantrain": _plain_scan, "scanstep": _plain_scanstep, "conv": _plain_conv,
                "convtrain": _plain_conv, "convstep": _plain_convstep, "ffn": _plain_ffn, "ffntrain": _plain_ffn}[op](s)
    from selective_state_space_ssd_gb300 import binding

    cu = s.get("cu")
    if op == "scan":
        y, final = binding.glr_forward(s["x"], s["r"], s["i"], s["lam"], h0=s.get("h0"), scale=C, cu_seqlens=cu)
        return dict(y=y, h_final=final)
    if op == "scantrain":
        stash = binding.glr_stash(s["x"])
        y, _ = binding.glr_forward(s["x"], s["r"], s["i"], s["lam"], h0=s.get("h0"), scale=C, cu_seqlens=cu, stash=stash)
        g = binding.glr_backward(s["dy"], s["x"], s["r"], s["i"], s["lam"], h0=s.get("h0"), scale=C, cu_seqlens=cu,
                                 stash=stash)
        out = dict(y=y, dx=g["dx"], dr=g["dr"], di=g["di"], dlam=g["dlam"])
        if "h0" in s:
            out["dh0"] = g["dh0"]
        return out
    if op == "scanstep":
        y = binding.glr_step(s["x"], s["r"], s["i"], s["lam"], s["state"], s["slots"], scale=C)
        return dict(y=y, state=s["state"])
    if op == "conv":
        y, taps = binding.conv_forward(s["x"], s["w"], s["b"], activation="silu", taps=s.get("taps"), cu_seqlens=cu)
        return dict(y=y, taps=taps)
    if op == "convtrain":
        y, _ = binding.conv_forward(s["x"], s["w"], s["b"], activation="silu")
        g = binding.conv_backward(s["dy"], s["x"], s["w"], s["b"], activation="silu")
        return dict(y=y, dx=g["dx"], dw=g["dw"], db=g["db"])
    if op == "convstep":
        y = binding.conv_step(s["x"], s["w"], s["b"], s["state"], s["slots"], activation="silu")
        return dict(y=y, state=s["state"])
    if op == "ffn":
        return dict(h=binding.ffn_forward(s["x"], s["wg"], s["wu"], activation=s["case"]["act"]))
    stash = binding.ffn_stash(s["x"], s["wg"])
    h = binding.ffn_forward(s["x"], s["wg"], s["wu"], activation=s["case"]["act"], stash=stash)
    g = binding.ffn_backward(s["dh"], s["x"], s["wg"], s["wu"], activation=s["case"]["act"], stash=stash)
    return dict(h=h, dx=g["dx"], dwg=g["dwg"], dwu=g["dwu"])


# ------------------------------------------------------------------------------------------------ the definition, 64 bits
def _spans(s):
    """(sequence, first step, last step + 1) of each sequence, over the steps of all batches on one axis."""
    n, t = s["case"]["N"], s["case"]["T"]
    lengths = s.get("lengths") or [t] * n
    begin = [0]
    for length in lengths:
        begin.append(begin[-1] + length)
    return [(j, begin[j], begin[j + 1]) for j in range(n)]


def _walked(s, a, b, first):
    """h after each step of every sequence, all sequences a step at a time; a, b [steps, D], first [N, D]."""
    spans = _spans(s)
    begin = torch.tensor([f for _, f, _ in spans], device="cuda")
    length = torch.tensor([e - f for _, f, e in spans], device="cuda")
    order = torch.argsort(length, descending=True)
    counts = sorted((e - f for _, f, e in spans), reverse=True)
    h = first.clone()
    out = torch.empty_like(b)
    alive = len(counts)
    for t in range(counts[0] if counts else 0):
        while alive and counts[alive - 1] <= t:
            alive -= 1
        who = order[:alive]
        at = begin[who] + t
        h[who] = a[at] * h[who] + b[at]
        out[at] = h[who]
    return out, h


def _exact_scan(s):
    case, d = s["case"], s["case"]["D"]
    flat = lambda z: z.double().reshape(-1, d)  # noqa: E731
    shape = s["x"].shape
    x, r, i, lam = flat(s["x"]), flat(s["r"]), flat(s["i"]), s["lam"].double()
    h0 = s["h0"].double() if "h0" in s else x.new_zeros(case["N"], d)

    def parts(x, r, i, lam):
        a = (1 + lam.exp()) ** (-C / (1 + torch.exp(-r)))
        return a, torch.sqrt((1 - a) * (1 + a)) * x / (1 + torch.exp(-i))

    a, b = parts(x, r, i, lam)
    h, last = _walked(s, a, b, h0)
    if case["op"] == "scan":
        return dict(y=h.reshape(shape), h_final=last)
    spans = [z for z in _spans(s) if z[2] > z[1]]
    before = torch.cat([x.new_zeros(1, d), h[:-1]])
    starts = torch.tensor([f for _, f, _ in spans], device="cuda")
    seqs = torch.tensor([j for j, _, _ in spans], device="cuda")
    before[starts] = h0[seqs]
    # the upstream gradients, walked from each sequence's end: what a step hands on is a times what it got
    dh = flat(s["dy"]).clone()
    ends = torch.tensor([e for _, _, e in spans], device="cuda")
    for t in range(1, max(e - f for _, f, e in spans)):
        at = ends[ends - starts > t] - 1 - t
        dh[at] += a[at + 1] * dh[at + 1]
    del h
    leaves = [z.clone().requires_grad_() for z in (x, r, i, lam)]
    with torch.enable_grad():
        a2, b2 = parts(*leaves)
        dx, dr, di, dlam = torch.autograd.grad((dh * (a2 * before + b2)).sum(), leaves)
    out = dict(y=None, dx=dx.reshape(shape), dr=dr.reshape(shape), di=di.reshape(shape), dlam=dlam)
    out["y"] = _walked(s, a, b, h0)[0].reshape(shape)
    if "h0" in s:
        out["dh0"] = torch.zeros_like(h0)
        out["dh0"][seqs] = a[starts] * dh[starts]
    return out


def _exact_conv(s):
    case, k = s["case"], s["case"]["K"]
    n, d = case["N"], case["D"]
    x, w, b = (s[z].double() for z in ("x", "w", "b"))
    x = x.reshape(-1, d)
    leaves = [z.clone().requires_grad_() for z in (x, w, b)]
    ys, last = [], []
    with torch.set_grad_enabled(case["op"] == "convtrain"):
        for j, f, e in _spans(s):
            head = s["taps"][j].double() if "taps" in s else x.new_zeros(k - 1, d)
            row = torch.cat([head, leaves[0][f:e]])
            z = leaves[2] + sum(leaves[1][:, m] * row[m:m + e - f] for m in range(k))
            ys.append(z / (1 + torch.exp(-z)))
            last.append(row[row.shape[0] - (k - 1):])
        y = torch.cat(ys).reshape(s["x"].shape)
        if case["op"] == "conv":
            return dict(y=y, taps=torch.stack(last))
        dx, dw, db = torch.autograd.grad(y, leaves, s["dy"].double())
    return dict(y=y.detach(), dx=dx.reshape(s["x"].shape), dw=dw, db=db)


def _exact_step(s):
    at = s["slots"].long()
    x, full = s["x"].double(), s["state"].double()
    if s["case"]["op"] == "scanstep":
        h, out = full[at], []
        for t in range(x.shape[1]):
            a = (1 + s["lam"].double().exp()) ** (-C / (1 + torch.exp(-s["r"][:, t].double())))
            h = a * h + torch.sqrt((1 - a) * (1 + a)) * x[:, t] / (1 + torch.exp(-s["i"][:, t].double()))
            out.append(h)
        full[at] = h
    else:
        row, out, k = torch.cat([full[at], x], 1), [], s["case"]["K"]
        for t in range(x.shape[1]):
            z = s["b"].double()
            for j in range(k):
                z = z + s["w"][:, j].double() * row[:, t + j]
            out.append(z / (1 + torch.exp(-z)))
        full[at] = row[:, row.shape[1] - (k - 1):]
    return dict(y=torch.stack(out, 1), state=full)


def exact(case, seed):
    op = case["op"]
    if op in ("ffn", "ffntrain") and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if op in ("scan", "scantrain"):
        return _exact_scan(s)
    if op in ("conv", "convtrain"):
        return _exact_conv(s)
    if op in ("scanstep", "convstep"):
        return _exact_step(s)
    leaves = [s[z].double().requires_grad_() for z in ("x", "wg", "wu")]
    with torch.set_grad_enabled(op == "ffntrain"):
        x, wg, wu = leaves
        g = x @ wg.T
        if case["act"] == "silu":
            act = g / (1 + torch.exp(-g))
        else:
            act = g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
        h = act * (x @ wu.T)
        if op == "ffn":
            return dict(h=h)
        dx, dwg, dwu = torch.autograd.grad(h, leaves, s["dh"].double())
    return dict(h=h.detach(), dx=dx, dwg=dwg, dwu=dwu)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, d = case["op"], case["D"]
    if op in ("ffn", "ffntrain"):
        m, f = case["M"], case["F"]
        once = m * d + 2 * d * f + m * f
        if op == "ffn":
            return dict(bytes=2 * once, flops=4 * m * d * f)
        # read again by the backward pass: x, the weights; beside them dh, dx and the weights' gradients
        return dict(bytes=2 * (2 * once + m * d + 2 * d * f), flops=12 * m * d * f)
    e = 4 if case["io"] == "f32" else 2
    n, t = case["N"], case["T"]
    steps = t if case.get("packed") else n * t
    if op.startswith("scan"):
        ends = 4 * n * d * (2 if case.get("h0") or op == "scanstep" else 1)
        if op == "scantrain":
            return dict(bytes=11 * steps * d * e + (4 * 3 * n * d if case.get("h0") else 0) + 12 * d, flops=70 * steps * d)
        return dict(bytes=4 * steps * d * e + ends + 4 * d, flops=25 * steps * d)
    k, we = case["K"], 4 if case["weights"] == "f32" else 2
    ends = (k - 1) * n * d * e * (2 if case.get("taps") or op == "convstep" else 1)
    if op == "convtrain":
        return dict(bytes=5 * steps * d * e + 3 * (k + 1) * d * we, flops=(8 * k + 20) * steps * d)
    return dict(bytes=2 * steps * d * e + ends + (k + 1) * d * we, flops=(2 * k + 8) * steps * d)
