"""The backward over packed batches of short sequences: every chunk is cut (fewer than 64 steps), a block of the gradient
kernel takes several of them one after another, and its two copy warps wait twice a chunk for the copies of a cut one.

Widths that are not whole 16-byte pieces are copied element by element, the others by TMA, so the four combinations of
(K, V) are the four orders in which a chunk's two waits can end.  Bounds as in test_delta_gpu.py."""
import numpy as np
import pytest
import torch

from selective_state_space_ssd_gb300 import binding

from test_delta_gpu import TOL_B, TOL_F, cfg_of, check, cuda, make, oracle

pytestmark = pytest.mark.gpu

LENGTHS = [1 + (29 * i) % 63 for i in range(500)]


def pass_with_status(cfg, dev, cu, stash=None):
    """o, s_final and the gradients, and the two calls' device status words."""
    x = tuple(dev[n] for n in ("q", "k", "v", "g", "beta"))
    prob = binding.delta_problem(cfg, packed=True)
    wf, wb = (torch.empty(binding.ssd_delta_workspace_size(prob, b, stash is not None), dtype=torch.uint8, device="cuda")
              for b in (False, True))
    o, sf = binding.delta_forward(cfg, *x, s0=dev["s0"], cu_seqlens=cu, stash=stash, workspace=(wf, wf.numel()))
    out = binding.delta_backward(cfg, dev["do"], *x, ds_final=dev["ds_final"], s0=dev["s0"], cu_seqlens=cu, stash=stash,
                                 workspace=(wb, wb.numel()))
    words = binding.ssd_read_status(wf), binding.ssd_read_status(wb)
    return dict(out, o=o, s_final=sf), words


@pytest.mark.parametrize("stashed", [False, True])
@pytest.mark.parametrize("K,V", [(20, 100), (128, 100), (20, 64), (128, 128), (64, 36), (100, 8)])
def test_many_cut_chunks_a_block(K, V, stashed):
    cfg = cfg_of(b=len(LENGTHS), T=sum(LENGTHS), H=2, HV=4, K=K, V=V)  # 1000 chunks and key heads on 152 blocks
    cpu = make(cfg, 41, packed=True)
    dev = cuda(cpu)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(LENGTHS)]), dtype=torch.int32)
    stash = binding.delta_stash(cfg, packed=True) if stashed else None
    got, words = pass_with_status(cfg, dev, cu.cuda(), stash)
    assert words == ((0, 0), (0, 0))
    again, words = pass_with_status(cfg, dev, cu.cuda(), stash)
    assert words == ((0, 0), (0, 0))
    for n in got:
        assert torch.equal(got[n], again[n]), n
    for i in range(0, len(LENGTHS), 17):
        a, length = int(cu[i]), LENGTHS[i]
        one = {k: (x[i:i + 1] if k in ("s0", "ds_final") else x[:, a:a + length]) for k, x in cpu.items()}
        ref = oracle(dict(cfg, batch=1, seqlen=length), one, K ** -0.5)
        check({k: (x[i:i + 1] if k in ("s_final", "ds0") else x[:, a:a + length]) for k, x in got.items()}, ref,
              {**TOL_F, **TOL_B})
