"""A gated-delta mixer block out of the library's operators: layer norm, the delta rule, layer norm of the heads.

    h = norm(x);   q, k, v, g, beta = projections of h;   o = delta rule(q, k, v, g, beta)
    y = x + W_o (norm over each head of o)

One set of weights serves three uses:

* :meth:`DeltaMixer.__call__`  whole sequences with gradients (training): the operators as autograd functions;
* :meth:`DeltaMixer.prefill`   packed prompts of any lengths, whose final states go into slots of a cache;
* :meth:`DeltaMixer.decode`    one or a few tokens of each running sequence, on the cache in place.

The projections and the keys' normalisation are plain torch; norms and delta rule run in the library's kernels.
``python -m selective_state_space_ssd_gb300.delta_mixer`` runs all three on small sizes.
"""
from __future__ import annotations

import torch

from . import binding


class FirstOrder(torch.autograd.Function):
    """Hands on the first `n` tensors, gradients that the library's kernels computed out of the others, and raises where
    they would be differentiated in their turn: taken for constants, they would drop terms without a word."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the library's gradients have no second derivative")


def first_order(grads, *of):
    """`grads` as a backward function returns them; a graph of them (create_graph) refuses to be used."""
    return FirstOrder.apply(len(grads), *grads, *of) if torch.is_grad_enabled() else grads


class LayerNorm(torch.autograd.Function):
    """``binding.norm_forward`` / ``binding.norm_backward`` on rows of the last dimension."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = binding.norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        g = binding.norm_backward(dy.contiguous(), x, mean, rstd, weight)
        of = (dy, x) if weight is None else (dy, x, weight)
        grads = first_order((g["dx"], g["dw"], g["db"]), *of)
        return *(t if need else None for t, need in zip(grads, ctx.needs_input_grad)), None


class DeltaRule(torch.autograd.Function):
    """``binding.delta_forward`` with its stash / ``binding.delta_backward``, from an empty first state.  ``status``: where
    both leave their device status word."""

    @staticmethod
    def forward(ctx, cfg, q, k, v, g, beta, status=None):
        stash = binding.delta_stash(cfg, q.device)
        o, _ = binding.delta_forward(cfg, q, k, v, g, beta, stash=stash, status=status)
        ctx.save_for_backward(q, k, v, g, beta, stash)
        ctx.cfg, ctx.status = cfg, status
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, g, beta, stash = ctx.saved_tensors
        d = binding.delta_backward(ctx.cfg, do.contiguous(), q, k, v, g, beta, stash=stash, status=ctx.status)
        return None, *first_order((d["dq"], d["dk"], d["dv"], d["dg"], d["dbeta"]), do, q, k, v, g, beta), None


class DeltaMixer:
    """Weights of one block (bf16 projections, fp32 norms and gate parameters), drawn from `seed`."""

    def __init__(self, width: int, nheads: int, value_heads: int, key_dim: int, value_dim: int, seed: int = 0,
                 device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        self.h, self.hv, self.kd, self.vd = nheads, value_heads, key_dim, value_dim
        self.parts = [nheads * key_dim, nheads * key_dim, value_heads * value_dim, value_heads, value_heads]
        p = dict(w_in=rn(sum(self.parts), width) * width ** -0.5,
                 w_out=rn(width, value_heads * value_dim) * (value_heads * value_dim) ** -0.5)
        p = {n: t.to(torch.bfloat16) for n, t in p.items()}
        p.update(norm_w=torch.ones(width), norm_b=torch.zeros(width), head_w=torch.ones(value_dim),
                 head_b=torch.zeros(value_dim), log_a=torch.rand(value_heads, generator=gen) * 2.0,
                 dt_bias=rn(value_heads) - 3.0)
        self.p = {n: t.to(device).requires_grad_() for n, t in p.items()}
        self.status = binding.delta_status(device)

    def check(self) -> None:
        """Waits for the block's calls so far and raises SSDError if a kernel of theirs gave up; a program does so where it
        waits for the GPU anyhow, once in so many steps."""
        try:
            binding.check_status(self.status)
        finally:
            self.status.zero_()

    def cfg(self, batch: int, seqlen: int) -> dict:
        return dict(dtype="bf16", gate_dtype="f32", batch=batch, seqlen=seqlen, nheads=self.h, value_heads=self.hv,
                    key_dim=self.kd, value_dim=self.vd)

    def inputs(self, h):
        """The delta rule's inputs from normed rows h [b, T, width]: q and k of unit length, log-decays, write gates."""
        q, k, v, a, b = (h @ self.p["w_in"].T).split(self.parts, dim=-1)
        unit = lambda x: torch.nn.functional.normalize(x.unflatten(-1, (self.h, self.kd)).float(), dim=-1).to(x.dtype)  # noqa: E731
        g = -torch.exp(self.p["log_a"]) * torch.nn.functional.softplus(a.float() + self.p["dt_bias"])
        return unit(q), unit(k), v.unflatten(-1, (self.hv, self.vd)), g.contiguous(), torch.sigmoid(b.float()).contiguous()

    def output(self, x, o, norm):
        o = norm(o, self.p["head_w"], self.p["head_b"], 1e-5)
        return x + o.flatten(-2) @ self.p["w_out"].T

    def __call__(self, x):
        """x [b, T, width] (bf16) to y, with gradients of x and of the weights."""
        h = LayerNorm.apply(x, self.p["norm_w"], self.p["norm_b"], 1e-5)
        q, k, v, g, beta = self.inputs(h)
        o = DeltaRule.apply(self.cfg(x.shape[0], x.shape[1]), q, k, v.contiguous(), g, beta, self.status)
        return self.output(x, o, LayerNorm.apply)

    @torch.no_grad()
    def prefill(self, x, cu_seqlens, state, slots):
        """Packed prompts x [tokens, width] with bounds cu_seqlens (int32) to y; prompt n's final state goes to
        state[slots[n]] of the cache [slots, HV, K, V], or nowhere if slots[n] is none of its slots."""
        norm = lambda *a: binding.norm_forward(*a)[0]  # noqa: E731
        h = norm(x, self.p["norm_w"], self.p["norm_b"], 1e-5)
        q, k, v, g, beta = self.inputs(h[None])
        # (v as the projection left it: a slice of wider rows)
        o, final = binding.delta_forward(self.cfg(slots.numel(), x.shape[0]), q, k, v, g, beta, cu_seqlens=cu_seqlens,
                                         status=self.status)
        # A place without a slot writes what another place writes too (the cache's own content where no place has a slot),
        # so that nothing waits for the device to count them.
        held = (slots >= 0) & (slots < state.shape[0])
        place = torch.where(held, torch.arange(slots.numel(), device=slots.device), held.int().argmax())
        slot = slots[place].long().clamp(0, state.shape[0] - 1)
        state[slot] = torch.where(held.any(), final[place], state[slot])
        return self.output(x, o[0], norm)

    @torch.no_grad()
    def decode(self, x, state, slots):
        """The next tokens x [b, T, width] of the sequences in `slots` to y; their states are updated in place."""
        norm = lambda *a: binding.norm_forward(*a)[0]  # noqa: E731
        h = norm(x, self.p["norm_w"], self.p["norm_b"], 1e-5)
        q, k, v, g, beta = self.inputs(h)
        o = binding.delta_step(self.cfg(x.shape[0], x.shape[1]), q, k, v, g, beta, state, slots)
        return self.output(x, o, norm)


def main() -> None:
    gen = torch.Generator(device="cuda").manual_seed(1)
    mixer = DeltaMixer(width=256, nheads=2, value_heads=4, key_dim=64, value_dim=64)
    x = torch.randn((2, 300, 256), generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
    y = mixer(x)
    y.float().square().mean().backward()
    print("training step: y", tuple(y.shape), "|dx|", float(x.grad.float().norm()), "|dW_in|",
          float(mixer.p["w_in"].grad.float().norm()))
    lengths = [100, 7, 193]
    cu = torch.tensor([0, 100, 107, 300], dtype=torch.int32, device="cuda")
    state = torch.zeros((4, 4, 64, 64), device="cuda")
    slots = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    mixer.prefill(x.detach()[0], cu, state, slots)
    token = torch.randn((3, 1, 256), generator=gen, device="cuda").to(torch.bfloat16)
    for _ in range(4):
        token = mixer.decode(token, state, slots)
    print("prompts of", lengths, "tokens, four more tokens each: y", tuple(token.shape), "finite:",
          bool(token.isfinite().all()))
    mixer.check()


if __name__ == "__main__":
    main()
