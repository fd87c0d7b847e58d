"""A small language model of selective-scan layers, trained, prompted and decoded with the library's layer operators.

Each layer is x + out_proj(scan(conv(in_proj(norm(x))))): ssd_layer_norm, ssd_conv (whose silu output feeds the scan),
ssd_selective with the gate z, each with its gradient in training, each for whole prompts with rows of their own
lengths, and the convolution and the scan for single tokens with their states in slots of a pool.  The projections, the
embedding and the loss are torch's.

    python examples/selective_lm.py [--steps 60]

trains on sequences in which every token names the next but one (one table for the even places, one for the odd), then
prompts three rows of unlike lengths, decodes them token by token, and compares the logits with those of one pass over
each whole row.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import state_space_sequence_ssd_gb300 as ssd  # noqa: E402


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = ssd.ssd_layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        g = ssd.ssd_layer_norm_backward(*ctx.saved_tensors, dy.contiguous())
        return g["dx"], g["dweight"], g["dbias"], None


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return ssd.ssd_conv_forward(x, weight, bias, want_final=False)[0]

    @staticmethod
    def backward(ctx, dy):
        g = ssd.ssd_conv_backward(*ctx.saved_tensors, dy.contiguous())
        return g["dx"], g["dweight"], g["dbias"]


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, dt_bias, z):
        ctx.save_for_backward(x, dt, A, B, C, D, dt_bias, z)
        return ssd.ssd_selective_forward(x, dt, A, B, C, D, dt_bias=dt_bias, dt_softplus=True, z=z, want_final=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, dt, A, B, C, D, dt_bias, z = ctx.saved_tensors
        g = ssd.ssd_selective_backward(x, dt, A, B, C, D, dy.contiguous(), dt_bias=dt_bias, dt_softplus=True, z=z)
        return (g["dx"], g["ddt"], g["dA"], g["dB"].to(B.dtype), g["dC"].to(C.dtype), g["dD"], g["ddt_bias"], g["dz"])


class Layer(torch.nn.Module):
    def __init__(self, width, inner, dstate, rank, taps):
        super().__init__()
        self.inner, self.dstate, self.rank, self.taps = inner, dstate, rank, taps
        self.norm_weight, self.norm_bias = (torch.nn.Parameter(v) for v in (torch.ones(width), torch.zeros(width)))
        self.in_proj = torch.nn.Linear(width, 2 * inner, bias=False)
        self.conv_weight = torch.nn.Parameter((torch.rand(inner, taps) * 2 - 1) * taps ** -0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(inner))
        self.x_proj = torch.nn.Linear(inner, rank + 2 * dstate, bias=False)
        self.dt_proj = torch.nn.Linear(rank, inner, bias=False)
        start = torch.exp(torch.rand(inner) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        self.dt_bias = torch.nn.Parameter(torch.log(torch.expm1(start)))
        self.A_log = torch.nn.Parameter(torch.log(torch.arange(1.0, dstate + 1)).repeat(inner, 1))
        self.D = torch.nn.Parameter(torch.ones(inner))
        self.out_proj = torch.nn.Linear(inner, width, bias=False)

    def scan_inputs(self, x):
        """dt, B, C of the scan from the convolution's output; B and C as slices of one projection."""
        low, B, C = self.x_proj(x).split([self.rank, self.dstate, self.dstate], -1)
        return self.dt_proj(low), B.unflatten(-1, (1, self.dstate)), C.unflatten(-1, (1, self.dstate))

    def forward(self, h):
        x, z = self.in_proj(LayerNorm.apply(h, self.norm_weight, self.norm_bias, 1e-5)).chunk(2, -1)
        x = Conv.apply(x, self.conv_weight, self.conv_bias)
        dt, B, C = self.scan_inputs(x)
        return h + self.out_proj(Scan.apply(x, dt, -torch.exp(self.A_log), B, C, self.D, self.dt_bias, z))

    def pool(self, slots, like):
        """States for `slots` sequences: the convolution's last inputs and the scan's states."""
        return (like.new_zeros(slots, self.taps - 1, self.inner), like.new_zeros(slots, self.inner, self.dstate, dtype=torch.float32))

    def prompt(self, h, lengths, pool, slots):
        """Rows of their own lengths; leaves the states after each row's last token in its slot."""
        y, _, _ = ssd.ssd_layer_norm_forward(h, self.norm_weight, self.norm_bias, 1e-5)
        x, z = self.in_proj(y).chunk(2, -1)
        x, last = ssd.ssd_conv_forward(x, self.conv_weight, self.conv_bias, lengths=lengths)
        dt, B, C = self.scan_inputs(x)
        y, state = ssd.ssd_selective_forward(x, dt, -torch.exp(self.A_log), B, C, self.D, lengths=lengths, dt_bias=self.dt_bias,
                                             dt_softplus=True, z=z)
        pool[0][slots.long()], pool[1][slots.long()] = last, state
        return h + self.out_proj(y)

    def step(self, h, pool, slots):
        y, _, _ = ssd.ssd_layer_norm_forward(h, self.norm_weight, self.norm_bias, 1e-5)
        x, z = self.in_proj(y).chunk(2, -1)
        x = ssd.ssd_conv_step(x, self.conv_weight, self.conv_bias, pool[0], slots)
        dt, B, C = self.scan_inputs(x)
        y = ssd.ssd_selective_step(x, dt, -torch.exp(self.A_log), B, C, self.D, pool[1], slots, dt_bias=self.dt_bias,
                                   dt_softplus=True, z=z)
        return h + self.out_proj(y)


class Model(torch.nn.Module):
    def __init__(self, vocab=64, width=128, layers=2, inner=256, dstate=16, rank=8, taps=4):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, width)
        self.layers = torch.nn.ModuleList(Layer(width, inner, dstate, rank, taps) for _ in range(layers))
        self.head = torch.nn.Linear(width, vocab, bias=False)

    def forward(self, tokens):
        h = self.embed(tokens)
        for layer in self.layers:
            h = layer(h)
        return self.head(h)

    @torch.no_grad()
    def prompt(self, tokens, lengths, slots, npool):
        h = self.embed(tokens)
        pools = [layer.pool(npool, h) for layer in self.layers]
        for layer, pool in zip(self.layers, pools):
            h = layer.prompt(h, lengths, pool, slots)
        return self.head(h[torch.arange(len(tokens), device=h.device), lengths.long() - 1]), pools

    @torch.no_grad()
    def step(self, tokens, pools, slots):
        h = self.embed(tokens)
        for layer, pool in zip(self.layers, pools):
            h = layer.step(h, pool, slots)
        return self.head(h)


def batch(rows, length, tables, rand):
    """Sequences whose token t + 2 is tables[t % 2][token t]."""
    seq = [torch.randint(0, tables.shape[1], (rows,), generator=rand, device="cuda") for _ in range(2)]
    while len(seq) < length:
        seq.append(tables[len(seq) % 2][seq[-2]])
    return torch.stack(seq, 1)


def main(steps=60, seed=0, quiet=False):
    torch.manual_seed(seed)
    rand = torch.Generator(device="cuda")
    rand.manual_seed(seed)
    tables = torch.stack([torch.randperm(64, generator=rand, device="cuda") for _ in range(2)])
    model = Model().cuda()
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3)
    losses = []
    for i in range(steps):
        t = batch(32, 129, tables, rand)
        loss = torch.nn.functional.cross_entropy(model(t[:, :-1]).flatten(0, 1), t[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if not quiet and (i % 10 == 0 or i + 1 == steps):
            print(f"step {i:3d}  loss {losses[-1]:.3f}")
    # prompts of unlike lengths in slots of a pool of five, then single tokens
    whole = batch(3, 48, tables, rand)
    lengths = torch.tensor([40, 17, 1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    logits, pools = model.prompt(whole, lengths, slots, 5)
    with torch.no_grad():
        want = model(whole)
    row = torch.arange(3, device="cuda")
    off = (logits - want[row, lengths.long() - 1]).abs().max().item()
    for k in range(8):
        at = lengths.long() + k
        logits = model.step(whole[row, at], pools, slots)
        off = max(off, (logits - want[row, at]).abs().max().item())
    if not quiet:
        print(f"prompt and eight decoded tokens: logits within {off:.2g} of one pass over the whole rows")
    return losses, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    main(ap.parse_args().steps)
