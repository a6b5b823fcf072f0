"""A small sequence model over the voxels of a grid batch.

The voxels of every grid, in the batch's own order, are the tokens of one
sequence; the grids' voxel offsets are the sequences' offsets, so nothing is
padded.  A block is: norm with the residual stream's addition, rotary positions
by voxel coordinate, linear attention with a decay for each head, and a product
back.  The model learns where the next voxel lies, and then walks a grid voxel
by voxel from its states alone.

    python examples/voxel_sequence.py [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_voxel_grid_leaf_gb300 as tb  # noqa: E402
from sparse_voxel_grid_leaf_gb300 import synth  # noqa: E402


def voxel_coordinates(batch):
    """int32 [V, 3] coordinates of the batch's voxels in its voxel order, and int64 [B + 1] offsets of its grids."""
    bits = (batch.masks[:, :, None] >> torch.arange(64, device=batch.masks.device)) & 1
    leaf, bit = bits.flatten(1).nonzero(as_tuple=True)
    local = torch.stack([bit // 64, bit % 64 // 8, bit % 8], 1).int()
    counts = batch.voxel_counts
    offsets = torch.zeros(counts.numel() + 1, dtype=torch.int64, device=counts.device)
    torch.cumsum(counts, 0, out=offsets[1:])
    return batch.origins[leaf] + local, offsets


class Block(torch.nn.Module):
    def __init__(self, width, heads, dim):
        super().__init__()
        self.heads, self.dim = heads, dim
        self.norm = torch.nn.Parameter(torch.ones(width))
        self.qkv = torch.nn.Linear(width, 3 * heads * dim, bias=False)
        self.out = torch.nn.Linear(heads * dim, width, bias=False)
        self.register_buffer("decay", 1 - 2.0 ** -torch.linspace(2, 9, heads))
        self.register_buffer("frequencies", tb.rotary_frequencies(dim, base=1000.0, axes=3, device="cpu"))

    def turned(self, x, residual, at):
        y, h = tb.rms_norm(x, self.norm.to(x.dtype), residual)
        q, k, v = self.qkv(y).unflatten(1, (3, self.heads, self.dim)).unbind(1)
        q, k = tb.rotary(q, k, at, self.frequencies)
        return q, k, v, h

    def forward(self, x, residual, at, offsets, state=None, return_state=False):
        """All rows of all grids: (output, residual stream[, states after each grid])."""
        q, k, v, h = self.turned(x, residual, at)
        o, last = tb.linear_attention(q, k, v, self.decay.float(), offsets, state=state, return_state=return_state)
        return (self.out(o.flatten(1)), h) + ((last,) if return_state else ())

    def step(self, x, residual, at, state):
        """One new row of each stream; the states are updated in place."""
        q, k, v, h = self.turned(x, residual, at)
        o = tb.linear_attention_step(q, k, v, self.decay.float(), state)
        return self.out(o.flatten(1)), h


class Model(torch.nn.Module):
    def __init__(self, width=128, heads=4, dim=32, blocks=2):
        super().__init__()
        self.enter = torch.nn.Linear(3, width)
        self.blocks = torch.nn.ModuleList(Block(width, heads, dim) for _ in range(blocks))
        self.norm = torch.nn.Parameter(torch.ones(width))
        self.leave = torch.nn.Linear(width, 3)

    def embed(self, at):
        return self.enter((at.float() / 32).to(self.enter.weight.dtype))

    def head(self, x, residual):
        y, _ = tb.rms_norm(x, self.norm.to(x.dtype), residual)
        return self.leave(y).float()

    def forward(self, at, offsets, return_states=False):
        x = self.embed(at)
        residual, states = torch.zeros_like(x), []
        for b in self.blocks:
            x, residual, *last = b(x, residual, at, offsets, return_state=return_states)
            states += last
        return (self.head(x, residual), states) if return_states else self.head(x, residual)

    def step(self, at, states):
        x = self.embed(at)
        residual = torch.zeros_like(x)
        for b, s in zip(self.blocks, states):
            x, residual = b.step(x, residual, at, s)
        return self.head(x, residual)


def run(steps=40, workload="pr1_b2_res32", seed=0, say=print):
    """Trains for `steps`; returns the losses and how far the walk by single voxels is from the whole pass."""
    torch.manual_seed(seed)
    ijk, off = synth.make(workload)
    batch = tb.from_ijk(torch.from_numpy(ijk).cuda(), torch.from_numpy(off).cuda())
    at, offsets = voxel_coordinates(batch)
    model = Model().cuda().to(torch.bfloat16)
    for b in model.blocks:
        b.decay = b.decay.float()
    inner = torch.ones(at.shape[0], dtype=torch.bool, device="cuda")
    inner[offsets[1:] - 1] = False  # a grid's last voxel has no next one
    ahead = (torch.roll(at, -1, 0) - at).float().clamp(-8, 8) / 8
    adam = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for i in range(steps):
        loss = (model(at, offsets) - ahead)[inner].square().mean()
        adam.zero_grad(set_to_none=True)
        loss.backward()
        adam.step()
        losses.append(loss.item())
        if say and (i % 10 == 0 or i + 1 == steps):
            say("step %d: loss %.4f over %d voxels of %d grids" % (i, losses[-1], at.shape[0], offsets.numel() - 1))
    with torch.no_grad():
        # every grid's first voxels in one pass, the next ones one at a time for all grids together
        whole = model(at, offsets)
        start = int((offsets[1:] - offsets[:-1]).min()) // 2
        head = torch.cat([torch.arange(start, device="cuda") + o for o in offsets[:-1]])
        cut = torch.arange(offsets.numel(), device="cuda") * start
        _, states = model(at[head], cut, return_states=True)
        off_by = 0.0
        for t in range(start, start + 8):
            rows = offsets[:-1] + t
            got = model.step(at[rows], states)
            off_by = max(off_by, (got - whole[rows]).abs().max().item())
    if say:
        say("voxel by voxel: at most %.4f from the whole pass" % off_by)
    return losses, off_by


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__)
    p.add_argument("--steps", type=int, default=40)
    run(p.parse_args().steps)
