"""The mixer block (layer norm, delta rule, head norm) as it is used: its training step against the same block in plain
torch in fp32 with the delta rule step by step, and prompts plus single tokens against whole sequences.

Bounds: y carries a few bf16 roundings one after another (projections, norms, o): 2e-2 of its largest value beside x; the
gradients pass them twice, through sums over tokens: 3e-2 in 2-norm."""
import pytest
import torch

from selective_state_space_ssd_gb300.delta_mixer import DeltaMixer

pytestmark = pytest.mark.gpu


def plain(mixer, p, x):
    """The block in fp32: p and x are fp32 leaves."""
    ln = lambda t, w, b: torch.nn.functional.layer_norm(t, t.shape[-1:], w, b, 1e-5)  # noqa: E731
    h = ln(x, p["norm_w"], p["norm_b"])
    q, k, v, a, b = (h @ p["w_in"].T).split(mixer.parts, dim=-1)
    unit = lambda t: torch.nn.functional.normalize(t.unflatten(-1, (mixer.h, mixer.kd)), dim=-1)  # noqa: E731
    G = mixer.hv // mixer.h
    q, k = (unit(t).repeat_interleave(G, 2) for t in (q, k))
    v = v.unflatten(-1, (mixer.hv, mixer.vd))
    g = -torch.exp(p["log_a"]) * torch.nn.functional.softplus(a + p["dt_bias"])
    beta = torch.sigmoid(b)
    s = x.new_zeros((x.shape[0], mixer.hv, mixer.kd, mixer.vd))
    out = []
    for t in range(x.shape[1]):
        s = torch.exp(g[:, t])[..., None, None] * s
        r = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, None, :] @ s)[..., 0, :])
        s = s + k[:, t, :, :, None] * r[:, :, None, :]
        out.append(mixer.kd ** -0.5 * (q[:, t, :, None, :] @ s)[..., 0, :])
    o = ln(torch.stack(out, 1), p["head_w"], p["head_b"])
    return x + o.flatten(-2) @ p["w_out"].T


def make(seed=0):
    mixer = DeltaMixer(width=192, nheads=2, value_heads=4, key_dim=64, value_dim=48, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    return mixer, lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_training_step_matches_plain_torch():
    mixer, rn = make()
    x, dy = rn(2, 130, 192).requires_grad_(), rn(2, 130, 192)
    y = mixer(x)
    y.backward(dy)
    p = {n: t.detach().float().requires_grad_() for n, t in mixer.p.items()}
    xf = x.detach().float().requires_grad_()
    yf = plain(mixer, p, xf)
    yf.backward(dy.float())
    assert float((y.detach().float() - yf.detach()).abs().max()) <= 2e-2 * float(yf.detach().abs().max())
    assert rel(x.grad, xf.grad) <= 3e-2
    for n, t in p.items():
        assert rel(mixer.p[n].grad, t.grad) <= 3e-2, n


def test_prompts_and_tokens_match_whole_sequences():
    mixer, rn = make(3)
    lengths = [70, 1, 131]
    x = rn(3, 135, 192)
    with torch.no_grad():
        whole = [mixer(x[i:i + 1, :n + 4])[0].float() for i, n in enumerate(lengths)]
    packed = torch.cat([x[i, :n] for i, n in enumerate(lengths)])
    cu = torch.tensor([0, 70, 71, 202], dtype=torch.int32, device="cuda")
    state = torch.full((5, 4, 64, 48), float("nan"), device="cuda")
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda")
    y = mixer.prefill(packed, cu, state, slots).float()
    for i, n in enumerate(lengths):
        a = int(cu[i])
        assert float((y[a:a + n] - whole[i][:n]).abs().max()) <= 2e-2 * float(whole[i].abs().max())
    for t in range(4):
        nxt = torch.stack([x[i, n + t] for i, n in enumerate(lengths)])[:, None]
        y = mixer.decode(nxt, state, slots).float()
        for i, n in enumerate(lengths):
            assert float((y[i, 0] - whole[i][n + t]).abs().max()) <= 2e-2 * float(whole[i].abs().max())
    assert state[[0, 3]].isnan().all()  # the cache's other slots are untouched
