"""The device status word of the delta rule's Python calls, which make and drop their workspace themselves: a wait that gave
up is seen in the tensor that the caller hands in.  The word is set by the test, after the call's kernels: no wait runs
out here."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding
from selective_state_space_ssd_gb300.delta_mixer import DeltaMixer

from test_delta_gpu import cfg_of, cuda, make

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta")


@pytest.fixture
def codes(monkeypatch):
    """The codes that the next calls' kernels 'leave', by entry point."""
    left = {}
    for name in ("ssd_delta_forward", "ssd_delta_backward"):
        def call(*args, real=getattr(binding, name), name=name):
            real(*args)
            if left.get(name):
                args[-3][:4].view(torch.int32).fill_(left[name])
        monkeypatch.setattr(binding, name, call)
    return left


@pytest.mark.parametrize("side", [False, True])
def test_a_wait_that_gave_up_is_seen(codes, side):
    cfg = cfg_of(b=1, T=70, H=1, HV=2, K=16, V=16)
    dev = cuda(make(cfg, 51))
    x = tuple(dev[n] for n in NAMES)
    stream = torch.cuda.Stream() if side else None
    status = binding.delta_status()
    torch.cuda.synchronize()
    both = lambda st: (binding.delta_forward(cfg, *x, status=st, stream=stream),  # noqa: E731
                       binding.delta_backward(cfg, dev["do"], *x, status=st, stream=stream))

    def word():
        torch.cuda.synchronize()
        return int(status)

    both(status)
    assert word() == 0
    binding.check_status(status)
    for name, code in (("ssd_delta_forward", 43), ("ssd_delta_backward", 124)):
        status.zero_()
        torch.cuda.synchronize()
        codes[name] = code
        both(status)
        codes.clear()
        both(status)  # a later call that is well does not hide it
        assert word() == code
        with pytest.raises(binding.SSDError, match=str(code)) as e:
            binding.check_status(status)
        assert e.value.status == 7
    ws = torch.empty(binding.ssd_delta_workspace_size(binding.delta_problem(cfg), False), dtype=torch.uint8, device="cuda")
    status.zero_()
    torch.cuda.synchronize()
    codes["ssd_delta_forward"] = 13
    binding.delta_forward(cfg, *x, workspace=(ws, ws.numel()), status=status, stream=stream)
    assert word() == 13 and binding.ssd_read_status(ws) == (7, 13)


def test_refusals():
    cfg = cfg_of(T=8)
    x = tuple(cuda(make(cfg, 52))[n] for n in NAMES)
    for bad in (torch.zeros(1, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            binding.delta_forward(cfg, *x, status=bad)
        with pytest.raises(ValueError):
            binding.delta_backward(cfg, x[2], *x, status=bad)


def test_a_number_without_dimensions(codes):
    cfg = cfg_of(T=8)
    x = tuple(cuda(make(cfg, 54))[n] for n in NAMES)
    status = torch.zeros((), dtype=torch.int32, device="cuda")
    codes["ssd_delta_forward"] = 9
    binding.delta_forward(cfg, *x, status=status)
    assert status.shape == () and int(status) == 9


def test_in_a_graph(codes):
    cfg = cfg_of(T=40, K=16, V=16)
    x = tuple(cuda(make(cfg, 53))[n] for n in NAMES)
    status = binding.delta_status()
    binding.delta_forward(cfg, *x, status=status)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.delta_forward(cfg, *x, status=status)
    status.fill_(-1)
    graph.replay()
    assert int(status) == 0


def test_the_mixer_block_sees_it(codes):
    mixer = DeltaMixer(width=64, nheads=1, value_heads=1, key_dim=16, value_dim=16)
    x = torch.randn((1, 20, 64), device="cuda").to(torch.bfloat16).requires_grad_()
    mixer(x).float().sum().backward()
    mixer.check()
    cu, slots = torch.tensor([0, 20], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    uses = (("ssd_delta_forward", lambda: mixer(x)), ("ssd_delta_backward", lambda: mixer(x).float().sum().backward()),
            ("ssd_delta_forward", lambda: mixer.prefill(x.detach()[0], cu, torch.zeros((1, 1, 16, 16), device="cuda"), slots)))
    for name, use in uses:
        codes[name] = 5
        use()
        codes.clear()
        with pytest.raises(binding.SSDError):
            mixer.check()
        mixer.check()  # told once
