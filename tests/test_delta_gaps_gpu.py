"""Steps of a packed axis that belong to no sequence (an axis padded to a fixed length, bounds that start late): o and the
gradients are zero there, whatever the buffers and the inputs held, and the sequences' own steps are what they are alone."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

from test_delta_gpu import cfg_of, cuda, make

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta")
GRADS = ("dq", "dk", "dv", "dg", "dbeta")

BOUNDS = {
    "padded": [0, 20, 20, 90],
    "late_and_padded": [5, 20, 84, 90],
    "late": [37, 40, 40, 100],
    "one_step_each_side": [1, 2, 3, 99],
    "empty": [0, 0, 0, 0],
    "empty_within": [33, 33, 33, 33],
    "past_the_end": [200, 300, 400, 500],
    "whole": [0, 1, 65, 100],
}


def calls(cfg, dev, cu, stashed):
    """The two calls on outputs full of NaN; o, s_final and the gradients."""
    prob = binding.delta_problem(cfg, packed=True)
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    out = dict(o=nan(dev["v"]), s_final=nan(dev["s0"]), ds0=nan(dev["s0"]), **{"d" + n: nan(dev[n]) for n in NAMES})
    stash = binding.delta_stash(cfg, packed=True) if stashed else None
    sb = stash.numel() if stashed else 0
    wf, wb = (torch.full((binding.ssd_delta_workspace_size(prob, b, stashed),), 255, dtype=torch.uint8, device="cuda")
              for b in (False, True))
    x = [dev[n] for n in NAMES]
    binding.ssd_delta_forward(prob, *x, dev["s0"], cu, 0.25, out["o"], out["s_final"], stash, sb, wf, wf.numel())
    binding.ssd_delta_backward(prob, dev["do"], dev["ds_final"], *x, dev["s0"], cu, 0.25, *(out[n] for n in GRADS), out["ds0"],
                               stash, sb, wb, wb.numel())
    assert binding.ssd_read_status(wf) == binding.ssd_read_status(wb) == (0, 0)
    return out


@pytest.mark.parametrize("stashed", [False, True])
@pytest.mark.parametrize("name", sorted(BOUNDS))
@pytest.mark.parametrize("sizes", [dict(H=1, HV=1, K=1, V=1, gates="bf16"), dict(H=1, HV=3, K=20, V=9),
                                   dict(H=2, HV=4, K=64, V=48, gates="bf16")])
def test_steps_of_no_sequence(sizes, name, stashed):
    cfg = cfg_of(b=3, T=100, **sizes)
    dev = cuda(make(cfg, 61, packed=True))
    bounds = BOUNDS[name]
    a, b = min(bounds[0], 100), min(bounds[-1], 100)
    for n in NAMES + ("do",):  # what lies there is nobody's
        dev[n][:, :a] = float("nan")
        dev[n][:, b:] = float("nan")
    got = calls(cfg, dev, torch.tensor(bounds, dtype=torch.int32, device="cuda"), stashed)
    for n in ("o",) + GRADS:
        assert (got[n][:, :a] == 0).all() and (got[n][:, b:] == 0).all(), n
    if b > a:
        part = {n: (t if n in ("s0", "ds_final") else t[:, a:b].clone()) for n, t in dev.items()}  # (on 16 bytes)
        own = torch.tensor([c - a for c in bounds], dtype=torch.int32, device="cuda")
        alone = calls(dict(cfg, seqlen=b - a), part, own, stashed)
        for n, t in alone.items():
            assert t.isfinite().all() and torch.equal(t, got[n] if n in ("s_final", "ds0") else got[n][:, a:b]), n
    else:
        assert torch.equal(got["s_final"], dev["s0"]) and torch.equal(got["ds0"], dev["ds_final"])


def test_a_long_padding():
    cfg = cfg_of(b=2, T=70001, H=2, HV=6, K=40, V=33)
    dev = cuda(make(cfg, 62, packed=True))
    got = calls(cfg, dev, torch.tensor([3, 100, 151], dtype=torch.int32, device="cuda"), False)
    for n in ("o",) + GRADS:
        assert (got[n][:, :3] == 0).all() and (got[n][:, 151:] == 0).all() and got[n][:, 3:151].isfinite().all(), n
