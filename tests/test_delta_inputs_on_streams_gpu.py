"""Inputs of a call on another stream than their own: freed on return, their memory must not go to the current stream's work
while the kernels on the other stream have yet to read it."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

from test_delta_gpu import cfg_of

pytestmark = pytest.mark.gpu
B, T = 2, 3000
CFG = cfg_of(b=B, T=T, H=1, HV=1, K=64, V=64)
STEP = cfg_of(b=3001, T=1, H=1, HV=1, K=64, V=64)


def bf(*s):
    return torch.full(s, 0.125, dtype=torch.bfloat16, device="cuda")


def delta_inputs(b, t):
    return dict(q=bf(b, t, 1, 64), k=bf(b, t, 1, 64), v=bf(b, t, 1, 64), g=torch.zeros((b, t, 1), device="cuda"),
                beta=torch.full((b, t, 1), 0.5, device="cuda"))


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


USES = {
    "delta_forward": (lambda: dict(delta_inputs(B, T), s0=torch.zeros((B, 1, 64, 64), device="cuda"), stash=binding.delta_stash(CFG)),
                      lambda s, x: binding.delta_forward(CFG, stream=s, **x)),
    "packed": (lambda: dict(delta_inputs(1, T), cu_seqlens=torch.tensor([0, 1000, T], dtype=torch.int32, device="cuda"),
                            status=status()),
               lambda s, x: binding.delta_forward(CFG, stream=s, **x)),
    "delta_backward": (lambda: dict(delta_inputs(B, T), dout=bf(B, T, 1, 64), ds_final=torch.zeros((B, 1, 64, 64), device="cuda"),
                                    s0=torch.zeros((B, 1, 64, 64), device="cuda")),
                       lambda s, x: binding.delta_backward(CFG, stream=s, **x)),
    "own_workspace": (lambda: dict(delta_inputs(B, T), w=torch.empty(
        binding.ssd_delta_workspace_size(binding.delta_problem(CFG), False), dtype=torch.uint8, device="cuda")),
        lambda s, x: binding.delta_forward(CFG, *(x[n] for n in ("q", "k", "v", "g", "beta")), stream=s,
                                           workspace=(x["w"], x["w"].numel()))),
    "delta_step": (lambda: dict(delta_inputs(3001, 1), state=torch.zeros((3001, 1, 64, 64), device="cuda"),
                                slots=torch.arange(3001, dtype=torch.int32, device="cuda")),
                   lambda s, x: binding.delta_step(STEP, stream=s, **x)),
    "norm_forward": (lambda: dict(x=bf(3000, 320), weight=torch.ones(320, device="cuda"), bias=torch.ones(320, device="cuda")),
                     lambda s, x: binding.norm_forward(stream=s, **x)),
    "norm_backward": (lambda: dict(dy=bf(3000, 320), x=bf(3000, 320), mean=torch.zeros(3000, device="cuda"),
                                   rstd=torch.ones(3000, device="cuda"), weight=torch.ones(320, device="cuda")),
                      lambda s, x: binding.norm_backward(stream=s, **x)),
}


@pytest.mark.parametrize("name", sorted(USES))
def test_inputs_stay_until_the_stream_has_read_them(name):
    make, call = USES[name]
    side = torch.cuda.Stream()
    call(side, make())  # (the first use of the stream and its memory)
    torch.cuda.synchronize()
    x = make()
    torch.cuda.synchronize()
    held = {n: (t.data_ptr(), t.numel() * t.element_size()) for n, t in x.items()}
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # some twenty milliseconds
    out = call(side, x)
    del x
    taken = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in held.values() for _ in range(4)]
    busy = not side.query()
    spans = [(t.data_ptr(), t.numel()) for t in taken]
    torch.cuda.synchronize()
    assert busy, "the other stream had finished: nothing was shown"
    bad = {n for n, (a, size) in held.items() for b, m in spans if a < b + m and b < a + size}
    assert not bad, bad
    del out
