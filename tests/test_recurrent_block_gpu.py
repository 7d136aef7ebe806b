"""The recurrent block (norm, convolution, recurrence, feed-forward) as it is used: its training step against the same block
in plain torch in fp32 with the recurrence step by step, and prompts plus single tokens against whole sequences.

Bounds: y carries a few bf16 roundings one after another (projections, norms, convolution, recurrence, feed-forward): 2e-2 of
its largest value; the gradients pass them twice, through sums over tokens: 3e-2 in 2-norm."""
import os
import subprocess
import sys

import pytest
import torch

from selective_state_space_ssd_gb300 import binding
from selective_state_space_ssd_gb300.recurrent_block import GatedFeedForward, Recurrence, RecurrentBlock, ShortConv

pytestmark = pytest.mark.gpu


def scan(x, r, i, lam, h):
    out = []
    for t in range(x.shape[1]):
        g = -8 * torch.nn.functional.softplus(lam) * torch.sigmoid(r[:, t])
        h = torch.exp(g) * h + torch.sqrt(-torch.expm1(2 * g)) * torch.sigmoid(i[:, t]) * x[:, t]
        out.append(h)
    return torch.stack(out, 1), h


def conv(x, w, b, taps=None):
    row = torch.cat([x.new_zeros((x.shape[0], w.shape[1] - 1, x.shape[2])) if taps is None else taps, x], 1)
    z = b + sum(w[:, j] * row[:, j:j + x.shape[1]] for j in range(w.shape[1]))
    return torch.nn.functional.silu(z), row[:, x.shape[1]:]


def plain(block, p, x):
    """The block in fp32: p and x are fp32 leaves."""
    ln = lambda t, w, b: torch.nn.functional.layer_norm(t, t.shape[-1:], w, b, 1e-5)  # noqa: E731
    u, z = (ln(x, p["norm_w"], p["norm_b"]) @ p["w_in"].T).split(block.inner, dim=-1)
    c, _ = conv(u, p["conv_w"], p["conv_b"])
    r, i = (c @ p["w_gates"].T).split(block.inner, dim=-1)
    s, _ = scan(c, r, i, p["lam"], x.new_zeros((x.shape[0], block.inner)))
    x = x + (s * torch.nn.functional.gelu(z, approximate="tanh")) @ p["w_out"].T
    h = ln(x, p["norm2_w"], p["norm2_b"])
    return x + (torch.nn.functional.silu(h @ p["w_ffn_gate"].T) * (h @ p["w_ffn_up"].T)) @ p["w_down"].T


def make(seed=0, width=192, inner=200, hidden=328):
    block = RecurrentBlock(width=width, inner=inner, hidden=hidden, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    return block, lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_training_step_matches_plain_torch():
    block, rn = make()
    x, dy = rn(2, 130, 192).requires_grad_(), rn(2, 130, 192)
    y = block(x)
    y.backward(dy)
    block.check()
    p = {n: t.detach().float().requires_grad_() for n, t in block.p.items()}
    xf = x.detach().float().requires_grad_()
    yf = plain(block, p, xf)
    yf.backward(dy.float())
    assert float((y.detach().float() - yf.detach()).abs().max()) <= 2e-2 * float(yf.detach().abs().max())
    assert rel(x.grad, xf.grad) <= 3e-2
    for n, t in p.items():
        assert rel(block.p[n].grad, t.grad) <= 3e-2, n


def test_prompts_and_tokens_match_whole_sequences():
    block, rn = make(3)
    lengths = [70, 1, 131]
    x = rn(3, 137, 192)
    with torch.no_grad():
        whole = [block(x[i:i + 1, :n + 6])[0].float() for i, n in enumerate(lengths)]
    packed = torch.cat([x[i, :n] for i, n in enumerate(lengths)])
    cu = torch.tensor([0, 70, 71, 202], dtype=torch.int32, device="cuda")
    cache = block.cache(5)
    for t in cache:
        t.fill_(float("nan"))
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    y = block.prefill(packed, cu, cache, slots).float()
    for i, n in enumerate(lengths):
        a = int(cu[i])
        assert float((y[a:a + n] - whole[i][:n]).abs().max()) <= 2e-2 * float(whole[i].abs().max())
    for t, few in ((0, 1), (1, 1), (2, 3), (5, 1)):  # single tokens, and a few at once
        nxt = torch.stack([x[i, n + t:n + t + few] for i, n in enumerate(lengths)])
        y = block.decode(nxt, cache, slots).float()
        for i, n in enumerate(lengths):
            assert float((y[i] - whole[i][n + t:n + t + few]).abs().max()) <= 2e-2 * float(whole[i].abs().max())
    assert all(t[[0, 3]].isnan().all() for t in cache)  # the cache's other slots are untouched


def test_places_without_a_slot_leave_the_cache():
    block, rn = make(5)
    x = rn(90, 192)
    cu = torch.tensor([0, 30, 80, 85, 90], dtype=torch.int32, device="cuda")
    full = block.cache(4)
    block.prefill(x, cu, full, torch.arange(4, dtype=torch.int32, device="cuda"))
    for slots, kept in (([-1, 1, 3, -7], {1: 1}), ([0, -1, 9, 2], {0: 0, 2: 3}), ([-1, 3, -1, -1], {})):
        cache = block.cache(3)
        for t in cache:
            t.fill_(0.5)
        at = torch.tensor(slots, dtype=torch.int32, device="cuda")
        block.prefill(x, cu, cache, at)
        for got, want in zip(cache, full):
            for s in range(3):
                assert torch.equal(got[s], want[kept[s]]) if s in kept else bool((got[s] == 0.5).all())
        assert block.decode(rn(4, 1, 192), cache, at).isfinite().all()


def test_sequences_in_two_pieces_have_the_same_gradients():
    """The taps and the state that a piece leaves carry its gradients."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, r, i, dy = (rn(2, 50, 40) for _ in range(4))
    w, b, lam = rn(40, 4), rn(40), rn(40) - 3

    def run(cuts):
        leaves = [t.clone().requires_grad_() for t in (x, r, i, w, b, lam)]
        xs, rs, gs, ws, bs, ls = leaves
        taps = h = None
        out = []
        for a, z in zip(cuts[:-1], cuts[1:]):
            c, taps = ShortConv.apply(xs[:, a:z].contiguous(), ws, bs, taps)
            s, h = Recurrence.apply(c, rs[:, a:z].contiguous(), gs[:, a:z].contiguous(), ls, h)
            out.append(s)
        y = torch.cat(out, 1)
        loss = (y * dy).sum() + h.sum() + taps.sum()
        return y.detach(), torch.autograd.grad(loss, leaves)

    whole = run([0, 50])
    for cuts in ([0, 23, 50], [0, 2, 3, 50], [0, 49, 50]):
        pieces = run(cuts)
        assert rel(pieces[0], whole[0]) <= 1e-5
        for a, c in zip(pieces[1], whole[1]):
            assert rel(a, c) <= 1e-5


@pytest.mark.parametrize("steps", [2, 9])
def test_one_sequence_without_a_batch_axis(steps):
    """The gradients of y, the taps and the state that follow, of [T, D] and of [1, T, D]: the same calls, the same bits."""
    _, rn = make(6)
    base, w, taps, dy, dl, ds = rn(steps, 24), rn(24, 4), rn(1, 3, 24), rn(steps, 24), rn(1, 3, 24), rn(1, 24).float()
    lam = torch.zeros(24, device="cuda")
    got = []
    for lead in ((), (1,)):
        x = base.reshape(*lead, steps, 24).clone().requires_grad_()
        k = taps.clone().requires_grad_()
        y, last = ShortConv.apply(x, w, None, k)
        s, h = Recurrence.apply(y, y, y, lam)
        got.append(torch.autograd.grad([s, last, h], [x, k], [dy.reshape(s.shape), dl, ds]))
    assert torch.equal(got[0][0], got[1][0][0]) and torch.equal(got[0][1], got[1][1])


def test_gradients_that_are_not_asked_for():
    gen = torch.Generator(device="cuda").manual_seed(8)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w = rn(1, 20, 24), rn(24, 3).requires_grad_()
    y, _ = ShortConv.apply(x, w)
    y.sum().backward()
    assert w.grad is not None and x.grad is None
    lam = rn(24).requires_grad_()
    _, last = Recurrence.apply(x, x, x, lam)
    last.sum().backward()  # only the final state is used
    assert lam.grad.isfinite().all()
    h = rn(16, 24).bfloat16()
    wg, wu = rn(32, 24).bfloat16().requires_grad_(), rn(32, 24).bfloat16()
    GatedFeedForward.apply(h, wg, wu).float().sum().backward()
    assert wg.grad is not None and wu.grad is None


@pytest.mark.parametrize("kind", ["conv", "scan", "ffn"])
def test_second_derivatives_are_refused(kind):
    gen = torch.Generator(device="cuda").manual_seed(9)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = rn(1, 20, 24).bfloat16().requires_grad_()
    y = {"conv": lambda: ShortConv.apply(x, rn(24, 3))[0], "scan": lambda: Recurrence.apply(x, x, x, rn(24))[0],
         "ffn": lambda: GatedFeedForward.apply(x, rn(32, 24).bfloat16(), rn(32, 24).bfloat16())}[kind]()
    first, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        first.float().square().sum().backward()


def calls(gen):
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, r, i, dy = (rn(2, 100, 64) for _ in range(4))
    lam, w, b = torch.rand(64, device="cuda") - 4, torch.randn((64, 4), generator=gen, device="cuda"), torch.zeros(64, device="cuda")
    h, wg, wu, dh = rn(200, 64), rn(96, 64), rn(96, 64), rn(200, 96)
    some = lambda d: tuple(t for t in d.values() if t is not None)  # noqa: E731
    return {"glr_forward": lambda s: binding.glr_forward(x, r, i, lam, stream=s),
            "glr_backward": lambda s: some(binding.glr_backward(dy, x, r, i, lam, stream=s)),
            "conv_forward": lambda s: binding.conv_forward(x, w, b, stream=s),
            "conv_backward": lambda s: some(binding.conv_backward(dy, x, w, b, stream=s)),
            "ffn_forward": lambda s: (binding.ffn_forward(h, wg, wu, stream=s),),
            "ffn_backward": lambda s: some(binding.ffn_backward(dh, h, wg, wu, stream=s)),
            "glr_step": lambda s: (binding.glr_step(x, r, i, lam, torch.zeros((2, 64), device="cuda"), stream=s),),
            "conv_step": lambda s: (binding.conv_step(x, w, b, torch.zeros((2, 3, 64), device="cuda", dtype=x.dtype), stream=s),)}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["glr_forward", "glr_backward", "conv_forward", "conv_backward", "ffn_forward",
                                  "ffn_backward"])
def test_call_on_another_stream(name, raw):
    """What a call allocates and frees must not be handed to the current stream's work while its kernels still use it."""
    call = calls(torch.Generator(device="cuda").manual_seed(11))[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(side)  # the first use of the stream and its memory
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
    got = call(side.cuda_stream if raw else side)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 9, 1 << 14, 1 << 18, 1 << 20, 3 << 20)
            for _ in range(8)]  # the current stream's work meanwhile, on memory that is free there
    torch.cuda.synchronize()
    assert len(junk) == 40
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    call = calls(torch.Generator(device="cuda").manual_seed(12))
    want = {n: f(None) for n, f in call.items()}
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [(n, f(s)) for _ in range(4) for s in streams for n, f in call.items()]
    torch.cuda.synchronize()
    for n, out in got:
        for a, b in zip(out, want[n]):
            assert torch.equal(a, b), n


def test_the_first_calls_of_a_process_can_be_captured():
    code = """
import torch
from selective_state_space_ssd_gb300 import binding as b
x = torch.randn((2, 200, 64), device="cuda").bfloat16()
lam, w = torch.zeros(64, device="cuda") - 4, torch.randn((64, 4), device="cuda")
wg = torch.randn((96, 64), device="cuda").bfloat16()
def calls():
    out = [*b.glr_forward(x, x, x, lam), *b.conv_forward(x, w), b.ffn_forward(x, wg, wg)]
    out += [b.glr_backward(x, x, x, x, lam)["dx"], b.conv_backward(x, x, w)["dx"], b.ffn_backward(out[-1], x, wg, wg)["dx"]]
    return out
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = calls()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, calls()))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
