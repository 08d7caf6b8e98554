"""A block around the linear-attention layer, trained and served: the layer's operators and
what surrounds them.

    x, residual -> residual addition and RMS norm             (gdn_add_norm_fwd / _bwd)
      -> one projection to q, k, v, gate
      -> q, k: RMS norm and the rotation by time, row, column (gdn_qk_norm_rope_axes_fwd / _bwd)
      -> linear attention with a decay for each head          (gdn_la_fwd / gdn_la_bwd / gdn_la_decode)
      -> gated RMS norm                                       (gdn_gated_norm_fwd / _bwd)
      -> output projection: the next block's x

Training clips the gradients' norm (gdn_clip_grads).  Serving takes the norm's output in 8 bits
with scales (gdn_add_norm_quant), parks the states of sequences that wait in 8 bits
(gdn_state_store) and resumes them (gdn_state_load).  Run on a GB300 after building the
library:

    python examples/linear_attention_block.py
"""
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from linear_attention_layer import GatedNorm, LinearAttention, gdn  # noqa: E402


class AddNorm(torch.autograd.Function):
    """(y, h) of x and the residual stream."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        y, h = gdn.gdn_add_norm_fwd(x, residual, weight)
        ctx.save_for_backward(h, weight)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        return gdn.gdn_add_norm_bwd(h, weight, dy.contiguous(), dh.contiguous())


class NormRopeAxes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions, sections):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        ctx.sections = sections
        return gdn.gdn_qk_norm_rope_axes_fwd(q, k, wq, wk, cos, sin, positions, sections)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        grads = gdn.gdn_qk_norm_rope_axes_bwd(*ctx.saved_tensors, ctx.sections, dq.contiguous(), dk.contiguous())
        return (*grads, None, None, None, None)


class Block(torch.nn.Module):
    def __init__(self, width, heads, dim, max_position, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.heads, self.dim = heads, dim
        new = dict(dtype=dtype, device=device)
        self.norm = torch.nn.Parameter(torch.ones(width, **new))
        self.project = torch.nn.Linear(width, 4 * heads * dim, bias=False, **new)
        self.out = torch.nn.Linear(heads * dim, width, bias=False, **new)
        # the query's scale 1 / sqrt(dim) lives in its norm's weight
        self.wq = torch.nn.Parameter(torch.full((dim,), dim ** -0.5, **new))
        self.wk = torch.nn.Parameter(torch.ones(dim, **new))
        self.wo = torch.nn.Parameter(torch.ones(dim, **new))
        h = torch.arange(1, heads + 1, dtype=torch.float32, device=device)
        self.register_buffer("log_decay", -torch.exp2(-8.0 * h / heads))
        angle = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * \
            10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64, device=device) * 2 / dim)
        self.register_buffer("cos", angle.cos().float())
        self.register_buffer("sin", angle.sin().float())
        side = dim // 2 * 3 // 8  # a quarter of the pairs for the time, the rest for row and column
        self.sections = (dim // 2 - 2 * side, side, side)

    def forward(self, x, residual, state, positions):
        """x, residual [B, T, width], positions [3, B, T]; returns the block's output, the
        residual stream behind its norm, and the state behind the last token."""
        y, h = AddNorm.apply(x, residual, self.norm)
        q, k, v, gate = self.project(y).unflatten(-1, (4, self.heads, self.dim)).unbind(-3)
        q, k = NormRopeAxes.apply(q, k, self.wq, self.wk, self.cos, self.sin, positions, self.sections)
        o, state = LinearAttention.apply(q, k, v, self.log_decay, state)
        return self.out(GatedNorm.apply(o, gate, self.wo).flatten(-2)), h, state

    @torch.no_grad()
    def step(self, x, residual, state, positions, eight_bits=True):
        """One token of every sequence; the state advances and the residual stream grows in
        place.  With `eight_bits` the projection reads the norm's output as e4m3 with a scale a
        row (multiplied out here; a product in 8 bits takes both as they are)."""
        if eight_bits:
            y8, scale, _ = gdn.gdn_add_norm_quant(x, residual, self.norm, h=residual)
            y = (y8.float() * scale).to(x.dtype)
        else:
            y, _ = gdn.gdn_add_norm_fwd(x, residual, self.norm, h=residual)
        q, k, v, gate = self.project(y).unflatten(-1, (4, self.heads, self.dim)).unbind(-3)
        q, k = gdn.gdn_qk_norm_rope_axes_fwd(q, k, self.wq, self.wk, self.cos, self.sin, positions, self.sections)
        o, _ = gdn.gdn_la_decode(q, k, v, self.log_decay, state)
        return self.out(gdn.gdn_gated_norm_fwd(o, gate, self.wo).flatten(-2))


def positions_of(batch, text, side, behind, device="cuda"):
    """Positions [3, batch, text + side * side + behind] of `text` tokens, one image of side x
    side, and `behind` more tokens of text."""
    t = torch.arange(text, device=device)
    i = torch.arange(side * side, device=device)
    image = torch.stack((torch.full_like(i, text), text + i // side, text + i % side))
    after = text + side + torch.arange(behind, device=device)
    p = torch.cat((t.expand(3, -1), image, after.expand(3, -1)), -1)
    return p[:, None].expand(3, batch, -1).to(torch.int32).contiguous()


class Model(torch.nn.Module):
    """Blocks on a residual stream in float32."""

    def __init__(self, depth=2, width=512, heads=4, dim=128, max_position=1024, dtype=torch.bfloat16):
        super().__init__()
        self.blocks = torch.nn.ModuleList(Block(width, heads, dim, max_position, dtype) for _ in range(depth))

    def new_states(self, batch):
        b = self.blocks[0]
        return [torch.zeros(batch, b.heads, b.dim, b.dim, device="cuda") for _ in self.blocks]

    def forward(self, x, states, positions):
        residual = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        ends = []
        for block, state in zip(self.blocks, states):
            x, residual, end = block(x, residual, state, positions)
            ends.append(end)
        return x + residual, ends

    @torch.no_grad()
    def step(self, x, states, positions, eight_bits=True):
        residual = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        for block, state in zip(self.blocks, states):
            x = block.step(x, residual, state, positions, eight_bits)
        return x + residual


def main(depth=2, width=512, heads=4, dim=128, batch=3, text=40, side=12, new_tokens=8, steps=10, max_norm=0.5, seed=0):
    torch.manual_seed(seed)
    positions = positions_of(batch, text, side, text + new_tokens)
    tokens = positions.shape[-1] - new_tokens
    model = Model(depth, width, heads, dim, int(positions.max()) + 1)
    optimiser = torch.optim.SGD(model.parameters(), lr=0.1)
    x = torch.randn(batch, tokens, width, device="cuda", dtype=torch.bfloat16)
    target = torch.nn.functional.pad(x, (0, 0, 1, 0))[:, :-1]
    norms = []
    for _ in range(steps):
        y, _ = model(x, model.new_states(batch), positions[..., :tokens].contiguous())
        loss = (y - target).float().square().mean()
        optimiser.zero_grad()
        loss.backward()
        norms.append(gdn.gdn_clip_grads([p.grad for p in model.parameters()], max_norm))
        optimiser.step()
    print(f"training on {batch} x {tokens} tokens: gradients of norm {float(norms[0]):.3f} to {float(norms[-1]):.3f}, "
          f"clipped to {max_norm}")

    # serving: a prompt; its sequences wait in a cache of 8-bit states while others could run; then
    # token by token, in another order, against the same without the wait
    more = torch.randn(batch, new_tokens, width, device="cuda", dtype=torch.bfloat16)
    slots = torch.randperm(batch + 2, device="cuda")[:batch].to(torch.int32)
    order = torch.randperm(batch, device="cuda")
    with torch.no_grad():
        _, ends = model(x, model.new_states(batch), positions[..., :tokens].contiguous())
        resumed = []
        for state in ends:
            cache = torch.empty(batch + 2, heads, dim, dim, dtype=torch.int8, device="cuda")
            scales = torch.empty(batch + 2, heads, dim, device="cuda")
            gdn.gdn_state_store(state, slots, cache, scales)
            resumed.append(gdn.gdn_state_load(cache, scales, slots[order].contiguous()))
        kept = [state.clone() for state in ends]
        outs, refs = [], []
        for t in range(new_tokens):
            at = positions[..., tokens + t:tokens + t + 1]
            outs.append(model.step(more[order, t:t + 1].contiguous(), resumed, at[:, order].contiguous()))
            refs.append(model.step(more[:, t:t + 1].contiguous(), kept, at.contiguous(), eight_bits=False))

    def off(a, b):
        return float((a - b).float().norm() / b.float().norm())
    o_off, s_off = off(torch.cat(outs, 1), torch.cat(refs, 1)[order]), off(torch.stack(resumed), torch.stack(kept)[:, order])
    print(f"{new_tokens} tokens behind parked states and 8-bit norms: outputs off by {o_off:.1e}, states by {s_off:.1e}")
    return [float(n) for n in norms], o_off, s_off


if __name__ == "__main__":
    main()
