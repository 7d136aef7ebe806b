"""The mixer block's prompts and tokens on one cache, with places that hold no sequence."""
import pytest
import torch

from selective_state_space_ssd_gb300.delta_mixer import DeltaMixer

pytestmark = pytest.mark.gpu


def test_a_padded_batch_of_prompts_leaves_the_other_slots():
    mixer = DeltaMixer(width=96, nheads=1, value_heads=2, key_dim=32, value_dim=24, seed=2)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((90, 96), generator=gen, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 30, 80, 85, 90], dtype=torch.int32, device="cuda")
    cache = torch.randn((3, 2, 32, 24), generator=gen, device="cuda")
    full = torch.zeros((4, 2, 32, 24), device="cuda")
    mixer.prefill(x, cu, full, torch.arange(4, dtype=torch.int32, device="cuda"))
    for slots, kept in (([-1, 1, 3, -7], {1: 1}), ([0, -1, 9, 2], {0: 0, 2: 3}), ([-1, 3, -1, -1], {})):
        state = cache.clone()
        at = torch.tensor(slots, dtype=torch.int32, device="cuda")
        mixer.prefill(x, cu, state, at)
        for s in range(3):
            assert torch.equal(state[s], full[kept[s]] if s in kept else cache[s]), (slots, s)
        token = torch.randn((4, 1, 96), generator=gen, device="cuda").to(torch.bfloat16)
        before = state.clone()
        y = mixer.decode(token, state, at)
        assert y.isfinite().all()
        for s in range(3):
            assert torch.equal(state[s], before[s]) == (s not in kept), (slots, s)
