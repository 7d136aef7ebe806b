"""Calls on a stream of the caller's: what a call allocates and frees must not be handed to the current stream's work while
the kernels on the other stream still use it.  And tensors that are not on one CUDA device are refused."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding
from selective_state_space_ssd_gb300.configs import DELTA_CONFIGS

pytestmark = pytest.mark.gpu
CFG = dict(DELTA_CONFIGS["delta_bf16"], batch=1, seqlen=200, nheads=2, value_heads=4, key_dim=64, value_dim=64)


def tensors(device="cuda"):
    gen = torch.Generator().manual_seed(7)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = dict(q=rn(1, 200, 2, 64) / 8, k=rn(1, 200, 2, 64) / 8, v=rn(1, 200, 4, 64), dout=rn(1, 200, 4, 64))
    x = {n: t.to(torch.bfloat16) for n, t in x.items()}
    x.update(g=-torch.rand((1, 200, 4), generator=gen), beta=torch.rand((1, 200, 4), generator=gen))
    return {n: t.to(device) for n, t in x.items()}


def calls(x):
    ins = tuple(x[n] for n in ("q", "k", "v", "g", "beta"))
    rows = x["v"].reshape(-1, 64)
    w = torch.ones(64, device="cuda")
    _, mean, rstd = binding.norm_forward(rows, w, w)
    torch.cuda.synchronize()
    return {"delta_forward": lambda s: binding.delta_forward(CFG, *ins, stream=s),
            "delta_backward": lambda s: tuple(t for t in binding.delta_backward(CFG, x["dout"], *ins, stream=s).values()
                                              if t is not None),
            "norm_forward": lambda s: binding.norm_forward(rows, w, w, stream=s),
            "norm_backward": lambda s: tuple(binding.norm_backward(rows, rows, mean, rstd, w, stream=s).values())}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["delta_forward", "delta_backward", "norm_forward", "norm_backward"])
def test_call_on_another_stream(name, raw):
    call = calls(tensors())[name]
    want = call(None)
    side = torch.cuda.Stream()
    call(side)  # the first use of the stream and its memory
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
    got = call(side.cuda_stream if raw else side)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 9, 1 << 14, 1 << 18, 1 << 20, 3 << 20)
            for _ in range(8)]  # the current stream's work meanwhile, on memory that is free there
    torch.cuda.synchronize()
    assert len(junk) == 40 and torch.cuda.current_stream() != side
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_tensors_off_the_device_are_refused():
    x, host = tensors(), tensors("cpu")
    names = ("q", "k", "v", "g", "beta")
    for n in names:
        with pytest.raises(ValueError):
            binding.delta_forward(CFG, *(host[m] if m == n else x[m] for m in names))
        with pytest.raises(ValueError):
            binding.delta_step(CFG, *(host[m] if m == n else x[m] for m in names), torch.zeros((1, 4, 64, 64), device="cuda"))
    with pytest.raises(ValueError):
        binding.delta_forward(CFG, *(host[m] for m in names))
    with pytest.raises(ValueError):
        binding.delta_backward(CFG, host["dout"], *(x[m] for m in names))
    with pytest.raises(ValueError):
        binding.delta_step(CFG, *(x[m] for m in names), torch.zeros((1, 4, 64, 64)))
    rows = x["v"].reshape(-1, 64)
    with pytest.raises(ValueError):
        binding.norm_forward(rows.cpu())
    with pytest.raises(ValueError):
        binding.norm_forward(rows, torch.ones(64))
    y, mean, rstd = binding.norm_forward(rows)
    with pytest.raises(ValueError):
        binding.norm_backward(y, rows, mean.cpu(), rstd)


@pytest.mark.parametrize("name", ["delta_forward", "delta_backward", "norm_backward"])
def test_workspace_stays_with_the_callers_stream(name, monkeypatch):
    """While the other stream is busy, the current stream is not given the block that the call took as its workspace."""
    call, taken = calls(tensors())[name], []
    launch = getattr(binding, "ssd_" + name)

    def spy(*args):
        taken.append((args[-3].data_ptr(), args[-3].numel()))
        launch(*args)

    monkeypatch.setattr(binding, "ssd_" + name, spy)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    call(side)
    at, n = taken[0]
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all(not (b.data_ptr() < at + n and at < b.data_ptr() + n) for b in blocks)


def test_calls_in_a_graph():
    """A server's step and its norm captured once and replayed: the state moves on with every replay."""
    x = tensors()
    step = dict(CFG, seqlen=1, batch=3)
    q, k, v = (torch.empty((3, 1) + x[n].shape[2:], dtype=torch.bfloat16, device="cuda") for n in ("q", "k", "v"))
    g, beta = (torch.empty((3, 1, 4), device="cuda") for _ in range(2))
    state, w = torch.zeros((3, 4, 64, 64), device="cuda"), torch.ones(64, device="cuda")

    def at(t):
        for buf, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta")):
            buf.copy_(x[n][0, 3 * t:3 * t + 3][:, None])

    def run():
        return binding.norm_forward(binding.delta_step(step, q, k, v, g, beta, state), w, w)[0]

    want, expect = state.clone(), []
    at(0)
    run()  # (the first call of a size loads its kernels)
    state.zero_()
    for t in range(5):
        at(t)
        expect.append(run())
    want.copy_(state)
    state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    state.zero_()
    for t in range(5):
        at(t)
        graph.replay()
        assert torch.equal(y, expect[t])
    assert torch.equal(state, want)


def test_training_step_in_a_graph():
    x = tensors()
    ins = tuple(x[n] for n in ("q", "k", "v", "g", "beta"))
    stash = binding.delta_stash(CFG)

    def run():
        o, sf = binding.delta_forward(CFG, *ins, stash=stash)
        return (o, sf) + tuple(t for t in binding.delta_backward(CFG, x["dout"], *ins, stash=stash).values() if t is not None)

    want = [t.clone() for t in run()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
