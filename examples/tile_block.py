"""A cross-attention block on the tiles, between the split and the blend.

    python examples/tile_block.py [workload]        (tiny, small, medium, temporal; default small)

One denoising-style step: the latent is split, every tile's tokens attend to the states of a padded prompt, and the tile
outputs are blended back.  Then a few training steps of the block (its dropout on) towards a target latent's tiles.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import blend_tdp_tile_gb300 as tdp  # noqa: E402
import workloads as wk  # noqa: E402
from blend_tdp_tile_gb300.block import TileBlock  # noqa: E402


def run(name="small", steps=4, lr=0.05, log=print):
    """Returns (blended latent, losses)."""
    wl = wk.by_name(name)
    dt = torch.float32 if wl.dtype == "f32" else torch.bfloat16
    torch.manual_seed(0)
    plan = tdp.tdp_plan_create(wl.B, wl.F, wl.H, wl.W, wl.C, wl.dtype, wl.num_tiles, wl.overlap)
    X = torch.randn(wl.B, wl.F, wl.H, wl.W, wl.C, device="cuda").to(dt)
    P = torch.from_numpy(wk.make_gen_positions(wl)).cuda()
    Y, Q, mn, mx = tdp.alloc_split_outputs(plan, X.device)
    tdp.tdp_pos_bounds(plan, P, mn, mx)
    tdp.tdp_split(plan, X, P, mn, 1, Y, Q)
    rows = Y.view(-1, wl.C)

    # a prompt of 77 states in a buffer of 128: the rest is padding
    context, S = 4 * wl.C, 128
    states = torch.randn(wl.B, S, context, device="cuda").to(dt)
    mask = (torch.arange(S, device="cuda") < 77).expand(wl.B, S).contiguous()
    block = TileBlock(wl.C, heads=8, kv_heads=4, head_dim=32, context=context, groups=wl.C // 4, p=0.1, dtype=dt)

    block.eval()
    with torch.no_grad():
        out = block(plan, rows, states, mask)
    Z = torch.empty_like(X)
    tdp.tdp_blend(plan, out, Z)
    log(f"{name}: {plan.n_tiles} tiles, {rows.shape[0]} rows, blended latent std {float(Z.float().std()):.4f}")

    block.train()
    target = rows.roll(1, 0)
    rng = torch.tensor([1234, 0], dtype=torch.int64, device="cuda")
    losses = []
    for step in range(steps):
        loss = (block(plan, rows, states, mask, rng).float() - target.float()).square().mean()
        loss.backward()
        with torch.no_grad():
            for w in block.parameters():
                w -= lr * w.grad.to(w.dtype)
                w.grad = None
        rng[1] += 1                       # the next step draws another mask
        losses.append(float(loss.detach()))
        log(f"  step {step}: loss {losses[-1]:.5f}")
    return Z, losses


if __name__ == "__main__":
    np.random.seed(0)
    run(*sys.argv[1:2])
