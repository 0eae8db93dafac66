"""A block that attends to conditioning tokens at their positions, trained with 8-bit checkpoints and served in 8 bits.

    python examples/rotary_block.py [workload]        (tiny, small, medium, temporal; default small)

The latent is split and the conditioning tokens filtered; a few training steps of the block (dropout on, the normalised rows kept in 8
bits) towards a target latent's tiles; then one pass with the projections in 8 bits, beside one with the full ones, blended back.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import blend_tdp_tile_gb300 as tdp  # noqa: E402
import workloads as wk  # noqa: E402
from blend_tdp_tile_gb300.block import RotaryBlock  # noqa: E402


def run(name="small", steps=4, lr=0.05, log=print):
    """Returns (blended latent of the 8-bit pass, of the full one, the last step's gradients)."""
    wl = wk.by_name(name)
    dt = torch.float32 if wl.dtype == "f32" else torch.bfloat16
    torch.manual_seed(0)
    plan = tdp.tdp_plan_create(wl.B, wl.F, wl.H, wl.W, wl.C, wl.dtype, wl.num_tiles, wl.overlap)
    _, P, K = wk.make_inputs(wl)
    S = K.shape[2]
    tokens_plan = tdp.tdp_plan_create(wl.B, 1, 1, S, wl.C, wl.dtype, (1, 1, 1), (0, 0, 0))
    X = torch.randn(wl.B, wl.F, wl.H, wl.W, wl.C, device="cuda").to(dt)
    Pd, Kd = torch.from_numpy(P).cuda(), torch.from_numpy(K).cuda()
    Y, Q, mn, mx = tdp.alloc_split_outputs(plan, X.device)
    keep, idx, count, kcount, Kout = tdp.alloc_filter_outputs(plan, S, X.device)
    # global positions: the tokens' origin is the same for every tile
    tdp.tdp_split_filter(plan, X, Pd, Kd, S, 0, Y, Q, mn, mx, keep, idx, count, kcount, Kout)
    rows, context = Y.view(-1, wl.C), 4 * wl.C
    tokens = torch.randn(wl.B, S, context, device="cuda").to(dt)
    block = RotaryBlock(wl.C, heads=8, kv_heads=4, head_dim=32, context=context, pairs=(6, 5, 5), p=0.1, keep8=True, dtype=dt)

    target = rows.roll(1, 0)
    rng = torch.tensor([1234, 0], dtype=torch.int64, device="cuda")
    for step in range(steps):
        loss = (block(plan, rows, Q, tokens_plan, tokens, Kd, keep, rng).float() - target.float()).square().mean()
        loss.backward()
        grads = {n: w.grad for n, w in block.named_parameters()}
        with torch.no_grad():
            for w in block.parameters():
                w -= lr * w.grad.to(w.dtype)
                w.grad = None
        rng[1] += 1                       # the next step draws another mask
        log(f"  step {step}: loss {float(loss.detach()):.5f}")

    got = []
    with torch.no_grad():
        for in8 in (False, True):
            block = block.to_8bit(plan) if in8 else block.eval()
            Z = torch.empty_like(X)
            tdp.tdp_blend(plan, block(plan, rows, Q, tokens_plan, tokens, Kd, keep), Z)
            got.append(Z)
    off = float((got[1].float() - got[0].float()).norm() / (got[0].float() - X.float()).norm())
    log(f"{name}: {plan.n_tiles} tiles, {rows.shape[0]} rows, {S} tokens; the 8-bit pass is {off:.3f} of the block's share off the full one")
    return got[1], got[0], grads


if __name__ == "__main__":
    run(*sys.argv[1:2])
