"""A recurrent block out of the library's operators: layer norm, short convolution, gated linear recurrence, and the gated
feed-forward behind it.

    h = norm(x);  u, z = projections of h;  c = convolution(u);  r, i = projections of c;  s = recurrence(c, r, i)
    x <- x + W_o (s gelu(z));      y = x + W_d ffn(norm(x))

One set of weights serves three uses:

* :meth:`RecurrentBlock.__call__`  whole sequences with gradients (training): the operators as autograd functions;
* :meth:`RecurrentBlock.prefill`   packed prompts of any lengths, whose final states and taps go into slots of a cache;
* :meth:`RecurrentBlock.decode`    one or a few tokens of each running sequence, on the cache in place.

The projections around the operators are plain torch.  ``python -m selective_state_space_ssd_gb300.recurrent_block`` runs
all three on small sizes.
"""
from __future__ import annotations

import torch

from . import binding
from .delta_mixer import LayerNorm, first_order


def first_orders(grads, *of):
    """``first_order`` of gradients some of which are None, out of tensors some of which are."""
    given = iter(first_order(tuple(g for g in grads if g is not None), *(t for t in of if t is not None)))
    return tuple(None if g is None else next(given) for g in grads)


class ShortConv(torch.autograd.Function):
    """``binding.conv_forward`` / ``binding.conv_backward`` on whole sequences [b, T, D] (or [T, D]): y and the taps that
    follow."""

    @staticmethod
    def forward(ctx, x, weight, bias=None, taps=None, activation="silu"):
        y, last = binding.conv_forward(x, weight, bias, activation, taps)
        ctx.save_for_backward(x, weight, bias, taps)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    def backward(ctx, dy, dlast):
        x, weight, bias, taps = ctx.saved_tensors
        dy = x.new_zeros(x.shape) if dy is None else dy.contiguous()
        g = binding.conv_backward(dy, x, weight, bias, ctx.activation, taps)
        dx, dtaps = g["dx"], g["dtaps"]
        if dlast is not None:  # the taps that follow are the last of the taps before and the inputs
            steps, held = x.shape[-2], dlast.shape[1]
            own = min(steps, held)
            dx.view(-1, *x.shape[-2:])[:, steps - own:] += dlast[:, held - own:]
            if dtaps is not None and own < held:
                dtaps.view(-1, *dtaps.shape[-2:])[:, own:] += dlast[:, :held - own]
        grads = first_orders((dx, g["dw"], g["db"], dtaps), dy, dlast, x, weight, bias, taps)
        return *(t if need else None for t, need in zip(grads, ctx.needs_input_grad)), None


class Recurrence(torch.autograd.Function):
    """``binding.glr_forward`` with its stash / ``binding.glr_backward`` on whole sequences: y and the final states."""

    @staticmethod
    def forward(ctx, x, r, i, lam, h0=None, scale=8.0):
        stash = binding.glr_stash(x)
        y, last = binding.glr_forward(x, r, i, lam, h0, scale, stash=stash)
        ctx.save_for_backward(x, r, i, lam, h0, stash)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    def backward(ctx, dy, dlast):
        x, r, i, lam, h0, stash = ctx.saved_tensors
        dy = x.new_zeros(x.shape) if dy is None else dy.contiguous()
        dlast = None if dlast is None else dlast.contiguous()
        g = binding.glr_backward(dy, x, r, i, lam, dlast, h0, ctx.scale, stash=stash)
        grads = first_orders((g["dx"], g["dr"], g["di"], g["dlam"], g["dh0"]), dy, dlast, x, r, i, lam, h0)
        return *(t if need else None for t, need in zip(grads, ctx.needs_input_grad)), None


class GatedFeedForward(torch.autograd.Function):
    """``binding.ffn_forward`` with its stash / ``binding.ffn_backward``.  ``status``: where both leave their device status
    word."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation="silu", status=None):
        stash = binding.ffn_stash(x, w_gate)
        h = binding.ffn_forward(x, w_gate, w_up, activation, stash=stash, status=status)
        ctx.save_for_backward(x, w_gate, w_up, stash)
        ctx.activation, ctx.status = activation, status
        return h

    @staticmethod
    def backward(ctx, dh):
        x, w_gate, w_up, stash = ctx.saved_tensors
        g = binding.ffn_backward(dh.contiguous(), x, w_gate, w_up, ctx.activation, stash=stash, status=ctx.status)
        grads = first_order((g["dx"], g["dwg"], g["dwu"]), dh, x, w_gate, w_up)
        return *(t if need else None for t, need in zip(grads, ctx.needs_input_grad)), None, None


class RecurrentBlock:
    """Weights of one block (bf16 projections; fp32 norms, convolution and decays), drawn from `seed`."""

    def __init__(self, width: int, inner: int, hidden: int, taps: int = 4, seed: int = 0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        self.width, self.inner, self.hidden, self.taps = width, inner, hidden, taps
        p = dict(w_in=rn(2 * inner, width) * width ** -0.5, w_gates=rn(2 * inner, inner) * inner ** -0.5,
                 w_out=rn(width, inner) * inner ** -0.5, w_ffn_gate=rn(hidden, width) * width ** -0.5,
                 w_ffn_up=rn(hidden, width) * width ** -0.5, w_down=rn(width, hidden) * hidden ** -0.5)
        p = {n: t.to(torch.bfloat16) for n, t in p.items()}
        decay = 0.9 + 0.099 * torch.rand(inner, generator=gen)  # of a step whose gate is open
        p.update(conv_w=rn(inner, taps) * taps ** -0.5, conv_b=torch.zeros(inner),
                 lam=torch.log(torch.expm1(-torch.log(decay) / 8.0)), norm_w=torch.ones(width), norm_b=torch.zeros(width),
                 norm2_w=torch.ones(width), norm2_b=torch.zeros(width))
        self.p = {n: t.to(device).requires_grad_() for n, t in p.items()}
        self.status = binding.delta_status(device)

    def check(self) -> None:
        """Waits for the block's calls so far and raises SSDError if a kernel of theirs gave up; a program does so where it
        waits for the GPU anyhow, once in so many steps."""
        try:
            binding.check_status(self.status)
        finally:
            self.status.zero_()

    def cache(self, slots: int) -> tuple:
        """An empty cache for so many sequences: their states [slots, inner] and taps [slots, taps - 1, inner]."""
        dev = self.p["lam"].device
        return (torch.zeros((slots, self.inner), device=dev),
                torch.zeros((slots, self.taps - 1, self.inner), dtype=torch.bfloat16, device=dev))

    def mix_in(self, h):
        """The convolution's input (a slice of the projection's wider rows) and the output's gate."""
        return (h @ self.p["w_in"].T).split(self.inner, dim=-1)

    def gates(self, c):
        return (c @ self.p["w_gates"].T).split(self.inner, dim=-1)

    def mix_out(self, x, s, z):
        return x + (s * torch.nn.functional.gelu(z, approximate="tanh")) @ self.p["w_out"].T

    def __call__(self, x):
        """x [b, T, width] (bf16) to y, with gradients of x and of the weights."""
        p = self.p
        u, z = self.mix_in(LayerNorm.apply(x, p["norm_w"], p["norm_b"], 1e-5))
        c, _ = ShortConv.apply(u, p["conv_w"], p["conv_b"])
        r, i = self.gates(c)
        s, _ = Recurrence.apply(c, r, i, p["lam"])
        x = self.mix_out(x, s, z)
        h = GatedFeedForward.apply(LayerNorm.apply(x, p["norm2_w"], p["norm2_b"], 1e-5), p["w_ffn_gate"], p["w_ffn_up"], "silu",
                                   self.status)
        return x + h @ p["w_down"].T

    def feed_forward(self, x):
        p = self.p
        h = binding.norm_forward(x, p["norm2_w"], p["norm2_b"], 1e-5)[0]
        return x + binding.ffn_forward(h, p["w_ffn_gate"], p["w_ffn_up"], status=self.status) @ p["w_down"].T

    @torch.no_grad()
    def prefill(self, x, cu_seqlens, cache, slots):
        """Packed prompts x [tokens, width] with bounds cu_seqlens (int32) to y; what prompt n leaves goes to slot slots[n] of
        the cache, or nowhere if that is none of its slots."""
        p, (state, taps) = self.p, cache
        u, z = self.mix_in(binding.norm_forward(x, p["norm_w"], p["norm_b"], 1e-5)[0])
        c, last = binding.conv_forward(u, p["conv_w"], p["conv_b"], cu_seqlens=cu_seqlens)
        r, i = self.gates(c)
        s, final = binding.glr_forward(c, r, i, p["lam"], cu_seqlens=cu_seqlens)
        # A place without a slot writes what another place writes too (the cache's own content where no place has a slot),
        # so that nothing waits for the device to count them.
        held = (slots >= 0) & (slots < state.shape[0])
        place = torch.where(held, torch.arange(slots.numel(), device=slots.device), held.int().argmax())
        slot = slots[place].long().clamp(0, state.shape[0] - 1)
        state[slot] = torch.where(held.any(), final[place], state[slot])
        taps[slot] = torch.where(held.any(), last[place], taps[slot])
        return self.feed_forward(self.mix_out(x, s, z))

    @torch.no_grad()
    def decode(self, x, cache, slots):
        """The next tokens x [b, T, width] of the sequences in `slots` to y; their states and taps are updated in place."""
        p, (state, taps) = self.p, cache
        u, z = self.mix_in(binding.norm_forward(x, p["norm_w"], p["norm_b"], 1e-5)[0])
        c = binding.conv_step(u, p["conv_w"], p["conv_b"], taps, slots)
        r, i = self.gates(c)
        s = binding.glr_step(c, r, i, p["lam"], state, slots)
        return self.feed_forward(self.mix_out(x, s, z))


def main() -> None:
    gen = torch.Generator(device="cuda").manual_seed(1)
    block = RecurrentBlock(width=256, inner=320, hidden=512)
    x = torch.randn((2, 300, 256), generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
    y = block(x)
    y.float().square().mean().backward()
    print("training step: y", tuple(y.shape), "|dx|", float(x.grad.float().norm()), "|dlam|", float(block.p["lam"].grad.norm()))
    cu = torch.tensor([0, 100, 107, 300], dtype=torch.int32, device="cuda")
    cache, slots = block.cache(4), torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    block.prefill(x.detach()[0], cu, cache, slots)
    token = torch.randn((3, 1, 256), generator=gen, device="cuda").to(torch.bfloat16)
    for _ in range(4):
        token = block.decode(token, cache, slots)
    print("prompts of [100, 7, 193] tokens, four more tokens each: y", tuple(token.shape), "finite:",
          bool(token.isfinite().all()))
    block.check()


if __name__ == "__main__":
    main()
