"""A linear-attention layer on the library's operators: training, a prompt, single tokens.

    x -> one projection to q, k, v, gate
      -> q, k: RMS norm of every head and the rotation   (gdn_qk_norm_rope_fwd / _bwd)
      -> linear attention with a decay for each head     (gdn_la_fwd / gdn_la_bwd / gdn_la_decode)
      -> RMS norm of every head times silu of the gate   (gdn_gated_norm_fwd / _bwd)
      -> output projection

The operators read q, k, v and the gate as slices of the projection's rows.  Run on a
GB300 after building the library:

    python examples/linear_attention_layer.py
"""
import math
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_delta_rule_19_gb300 import gdn  # noqa: E402


class NormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        return gdn.gdn_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        grads = gdn.gdn_qk_norm_rope_bwd(*ctx.saved_tensors, dq.contiguous(), dk.contiguous())
        return (*grads, None, None, None)


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, state):
        o, final, saved = gdn.gdn_la_fwd(q, k, v, log_decay, state, saved=True)
        ctx.save_for_backward(q, k, v, log_decay, state, saved)
        return o, final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o, d_final):
        *inputs, saved = ctx.saved_tensors
        dq, dk, dv, d_state = gdn.gdn_la_bwd(*inputs, d_o.contiguous(), d_final.contiguous(), saved=saved)
        return dq, dk, dv, None, d_state


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight):
        ctx.save_for_backward(x, gate, weight)
        return gdn.gdn_gated_norm_fwd(x, gate, weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return gdn.gdn_gated_norm_bwd(*ctx.saved_tensors, dy.contiguous())


class Layer(torch.nn.Module):
    def __init__(self, width, heads, dim, max_tokens, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.heads, self.dim = heads, dim
        new = dict(dtype=dtype, device=device)
        self.project = torch.nn.Linear(width, 4 * heads * dim, bias=False, **new)
        self.out = torch.nn.Linear(heads * dim, width, bias=False, **new)
        # the query's scale 1 / sqrt(dim) lives in its norm's weight
        self.wq = torch.nn.Parameter(torch.full((dim,), dim ** -0.5, **new))
        self.wk = torch.nn.Parameter(torch.ones(dim, **new))
        self.wo = torch.nn.Parameter(torch.ones(dim, **new))
        h = torch.arange(1, heads + 1, dtype=torch.float32, device=device)
        self.register_buffer("log_decay", -torch.exp2(-8.0 * h / heads))
        angle = torch.arange(max_tokens, dtype=torch.float64, device=device)[:, None] * \
            10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64, device=device) * 2 / dim)
        self.register_buffer("cos", angle.cos().float())
        self.register_buffer("sin", angle.sin().float())

    def new_state(self, batch):
        return torch.zeros(batch, self.heads, self.dim, self.dim, device=self.wq.device)

    def rows(self, x):
        r = self.project(x).unflatten(-1, (4, self.heads, self.dim))
        return r.unbind(-3)  # q, k, v, gate: slices, not copies

    def forward(self, x, state, positions):
        """x [B, T, width]; returns the outputs and the state behind the last token."""
        q, k, v, gate = self.rows(x)
        q, k = NormRope.apply(q, k, self.wq, self.wk, self.cos, self.sin, positions)
        o, state = LinearAttention.apply(q, k, v, self.log_decay, state)
        return self.out(GatedNorm.apply(o, gate, self.wo).flatten(-2)), state

    @torch.no_grad()
    def step(self, x, state, positions):
        """One token of every sequence, x [B, 1, width]; the state advances in place."""
        q, k, v, gate = self.rows(x)
        q, k = gdn.gdn_qk_norm_rope_fwd(q, k, self.wq, self.wk, self.cos, self.sin, positions)
        o, _ = gdn.gdn_la_decode(q, k, v, self.log_decay, state)
        return self.out(gdn.gdn_gated_norm_fwd(o, gate, self.wo).flatten(-2))


def positions_of(batch, first, count):
    t = torch.arange(first, first + count, dtype=torch.int32, device="cuda")
    return t.expand(batch, count).contiguous()


def main(width=512, heads=4, dim=128, batch=2, tokens=700, steps=20, new_tokens=16, seed=0):
    torch.manual_seed(seed)
    layer = Layer(width, heads, dim, tokens + new_tokens)
    # training: the layer learns to give back its input of one token earlier
    optimiser = torch.optim.Adam(layer.parameters(), lr=2e-3)
    x = torch.randn(batch, tokens, width, device="cuda", dtype=torch.bfloat16)
    target = torch.nn.functional.pad(x, (0, 0, 1, 0))[:, :-1]
    losses = []
    for _ in range(steps):
        y, _ = layer(x, layer.new_state(batch), positions_of(batch, 0, tokens))
        loss = (y - target).float().square().mean()
        optimiser.zero_grad()
        loss.backward()
        optimiser.step()
        losses.append(float(loss.detach()))
    print(f"training on {batch} x {tokens} tokens: loss {losses[0]:.3f} -> {losses[-1]:.3f}")

    # serving: a prompt in one call, then token by token, against one call over everything
    more = torch.randn(batch, new_tokens, width, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        every, last = layer(torch.cat([x, more], 1), layer.new_state(batch),
                            positions_of(batch, 0, tokens + new_tokens))
        _, state = layer(x, layer.new_state(batch), positions_of(batch, 0, tokens))
        state = state.clone()
        outs = [layer.step(more[:, t:t + 1], state, positions_of(batch, tokens + t, 1)) for t in range(new_tokens)]
    def off(a, b):
        return float((a - b).float().norm() / b.float().norm())
    o_off, s_off = off(torch.cat(outs, 1), every[:, tokens:]), off(state, last)
    print(f"{new_tokens} single tokens after the prompt: outputs off by {o_off:.1e}, state by {s_off:.1e} of one call's")
    return losses, o_off, s_off


if __name__ == "__main__":
    main()
