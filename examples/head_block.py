"""A small sequence model of head-scan blocks: training on a synthetic copy task, then decoding token by token.

    python examples/head_block.py [--steps 600]

Each block is
    out, r   = residual_norm(previous block's output, residual stream r)
    z, x, B, C, dt = in_proj(out)                 (views of one projection's rows: no copies)
    y        = head_scan(x, dt, A_log, B, C, D)
    previous block's output = out_proj(gated_norm(y, z))
in training and for the prompt; for each further token head_scan becomes head_state_update on the state that the
prompt left.  The projections and the optimizer are torch's.  Needs an MI355X and the built library.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_softplus_amd as ss  # noqa: E402


class HeadBlock(torch.nn.Module):
    def __init__(self, d_model, heads, head_dim, state, groups=1):
        super().__init__()
        self.H, self.P, self.N, self.G = heads, head_dim, state, groups
        self.d = heads * head_dim
        self.norm = torch.nn.Parameter(torch.ones(d_model))
        self.gate = torch.nn.Parameter(torch.ones(self.d))
        self.in_proj = torch.nn.Linear(d_model, 2 * self.d + 2 * groups * state + heads, bias=False)
        self.out_proj = torch.nn.Linear(self.d, d_model, bias=False)
        self.A_log = torch.nn.Parameter(torch.log(torch.linspace(1.0, 16.0, heads)))
        self.D = torch.nn.Parameter(torch.ones(heads))
        step = torch.exp(torch.rand(heads) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))

    def split(self, proj):
        z, x, B, C, dt = proj.split([self.d, self.d, self.G * self.N, self.G * self.N, self.H], -1)
        return (z, x.unflatten(-1, (self.H, self.P)), B.unflatten(-1, (self.G, self.N)),
                C.unflatten(-1, (self.G, self.N)), dt)

    def forward(self, h, r, state=None):
        """h: the previous block's output (b, L, d_model), r: the residual stream (fp32) or None.
        Returns this block's output, the stream and the last state."""
        out, r = ss.residual_norm(h, self.norm, residual=r, residual_dtype=torch.float32)
        z, x, B, C, dt = self.split(torch.nn.functional.linear(out, self.in_proj.weight.to(out.dtype)))
        y, last = ss.head_scan(x, dt, self.A_log, B, C, self.D, delta_bias=self.dt_bias, initial_state=state,
                               return_last_state=True)
        y = ss.gated_norm(y.flatten(-2), z, self.gate, groups=self.G)
        return torch.nn.functional.linear(y, self.out_proj.weight.to(y.dtype)), r, last

    @torch.no_grad()
    def step(self, h, r, state):
        """One token: h (b, d_model), r (b, d_model) or None; state (b, H, P, N) is updated in place."""
        out, r = ss.residual_norm_fwd(h, self.norm, residual=r, residual_dtype=torch.float32)
        z, x, B, C, dt = self.split(torch.nn.functional.linear(out, self.in_proj.weight.to(out.dtype)))
        y = ss.head_state_update(state, x.contiguous(), dt.contiguous(), self.A_log, B.contiguous(), C.contiguous(),
                                 self.D, dt_bias=self.dt_bias)
        y = ss.gated_norm_fwd(y.flatten(-2), z, self.gate, groups=self.G)
        return torch.nn.functional.linear(y, self.out_proj.weight.to(y.dtype)), r


class HeadModel(torch.nn.Module):
    def __init__(self, vocab=32, d_model=128, layers=2, heads=4, head_dim=64, state=64, dtype=torch.bfloat16):
        super().__init__()
        self.dtype = dtype
        self.embed = torch.nn.Embedding(vocab, d_model)
        torch.nn.init.normal_(self.embed.weight, std=0.05)   # also the output projection
        self.blocks = torch.nn.ModuleList(HeadBlock(d_model, heads, head_dim, state) for _ in range(layers))
        self.norm = torch.nn.Parameter(torch.ones(d_model))

    def head(self, h, r, norm):
        out, _ = norm(h, self.norm, residual=r)
        return torch.nn.functional.linear(out, self.embed.weight.to(out.dtype)).float()

    def forward(self, tokens, states=None):
        """Logits (b, L, vocab) and every block's last state."""
        h, r, last = self.embed(tokens).to(self.dtype), None, []
        for k, block in enumerate(self.blocks):
            h, r, s = block(h, r, None if states is None else states[k])
            last.append(s)
        return self.head(h, r, ss.residual_norm), last

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits (b, vocab) of one token each; the states are updated in place."""
        h, r = self.embed(tokens).to(self.dtype), None
        for block, state in zip(self.blocks, states):
            h, r = block.step(h, r, state)
        return self.head(h, r, ss.residual_norm_fwd)


def copy_task(b, length, vocab, generator, device):
    """`length` random tokens, a mark, and the same tokens again: the second half is predictable."""
    first = torch.randint(1, vocab, (b, length), generator=generator, device=device)
    mark = torch.zeros((b, 1), dtype=first.dtype, device=device)
    return torch.cat([first, mark, first], 1)


def train(model, steps, b=64, length=8, lr=3e-3, seed=0, report=None):
    """Losses over the predictable half, one a step."""
    device = next(model.parameters()).device
    gen = torch.Generator(device=device).manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for k in range(steps):
        tokens = copy_task(b, length, model.embed.num_embeddings, gen, device)
        logits, _ = model(tokens[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits[:, length:].flatten(0, 1), tokens[:, length + 1:].flatten())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if report and (k + 1) % report == 0:
            print(f"step {k + 1}: loss {losses[-1]:.4f}", flush=True)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=600)
    args = ap.parse_args()
    torch.manual_seed(0)
    model = HeadModel().to("cuda")
    train(model, args.steps, report=100)
    length = 8
    tokens = copy_task(64, length, 32, torch.Generator(device="cuda").manual_seed(1), "cuda")
    with torch.no_grad():
        logits, states = model(tokens[:, :length + 1])   # the prompt, up to the mark
        got = [logits[:, -1]]
        for k in range(length + 1, tokens.shape[1] - 1):     # then token by token
            got.append(model.step(tokens[:, k], states))
        right = (torch.stack(got, 1).argmax(-1) == tokens[:, length + 1:]).float().mean().item()
    print(f"copied tokens right while decoding: {right:.2f}", flush=True)


if __name__ == "__main__":
    main()
