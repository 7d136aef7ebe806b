"""Where a prompt's final state goes: places without a sequence (slots outside the cache) touch no state, as in the calls
of single tokens.  Plain tensor code on the CPU."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding, delta_mixer


@pytest.mark.parametrize("slots", [[2, 0, 3], [-1, 1, 2], [1, -1, 4], [4, 1 << 30, 0], [-1, -5, 4], [-(1 << 31), 3, (1 << 31) - 1]])
def test_prompts_without_a_slot_touch_no_state(slots, monkeypatch):
    gen = torch.Generator().manual_seed(1)
    mixer = delta_mixer.DeltaMixer(width=8, nheads=1, value_heads=2, key_dim=4, value_dim=3, device="cpu")
    final = torch.randn((3, 2, 4, 3), generator=gen)
    monkeypatch.setattr(binding, "norm_forward", lambda x, w, b, eps: (x, None, None))
    monkeypatch.setattr(binding, "delta_forward", lambda cfg, q, k, v, *a, **o: (v.contiguous(), final))
    cache = torch.randn((4, 2, 4, 3), generator=gen)
    cache[0] = float("nan")
    state, want = cache.clone(), cache.clone()
    for n, s in enumerate(slots):
        if 0 <= s < 4:
            want[s] = final[n]
    x = torch.randn((6, 8), generator=gen).to(torch.bfloat16)
    mixer.prefill(x, torch.tensor([0, 1, 5, 6], dtype=torch.int32), state, torch.tensor(slots, dtype=torch.int32))
    assert torch.equal(state.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(state.isnan(), want.isnan())
