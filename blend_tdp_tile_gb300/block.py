"""The per-tile block's operators as differentiable torch functions, and a block made of them.

Between ``tdp_split`` and ``tdp_blend`` a transformer runs on every tile.  The functions here
put the library's operators on tile-major rows under torch's autograd:

  group_norm(plan, x, groups, gamma, beta)   statistics of every (tile, item), channels last, SiLU
  cross_attn(plan, q, k, v, mask)            tile rows attend to an encoder's states
  dropout_add(plan, x, res, p, rng)          residual + dropout whose mask is never stored

``TileBlock`` is one cross-attention sublayer of them: normalise, project, attend, project back,
drop out and add.  All tiles go through each call at once; nothing is padded.  The gradients are first ones: a
derivative of theirs raises an error.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (Plan, tdp_cross_attn, tdp_cross_attn_grad, tdp_dropout_add, tdp_dropout_grad, tdp_group_norm,
               tdp_group_norm_grad)

__all__ = ["group_norm", "cross_attn", "dropout_add", "TileBlock"]


def _dense(t):
    """t as the library takes it: contiguous, on a 16-byte boundary (a cat's gradient starts anywhere)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, x, groups, gamma, beta, eps, act):
        x = _dense(x)
        stats = [torch.empty((plan.n_tiles, plan.B, groups), dtype=torch.float32, device=x.device) for _ in range(2)]
        y = torch.empty_like(x)
        tdp_group_norm(plan, x, groups, gamma, beta, y, *stats, eps=eps, act=act)
        ctx.plan, ctx.groups, ctx.act = plan, groups, act
        ctx.save_for_backward(x, gamma, beta, *stats)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, gamma, beta, mean, rstd = ctx.saved_tensors
        dx = torch.empty_like(x)
        params = gamma is not None or beta is not None
        dgamma, dbeta = (torch.empty(x.shape[-1], dtype=torch.float32, device=x.device) if params else None for _ in range(2))
        tdp_group_norm_grad(ctx.plan, x, ctx.groups, gamma, beta, mean, rstd, _dense(dy), dx, dgamma, dbeta, act=ctx.act)
        return (None, dx, None, None if gamma is None else dgamma.to(gamma.dtype),
                None if beta is None else dbeta.to(beta.dtype), None, None)


class _CrossAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, q, k, v, mask, scale):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        tdp_cross_attn(plan, q, k, v, mask, out, lse, scale=scale)
        ctx.plan, ctx.scale = plan, scale
        ctx.save_for_backward(q, k, v, mask, out, lse)      # the mask too: one refilled in between is an error
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, mask, out, lse = ctx.saved_tensors
        dq = torch.empty_like(out)
        dk, dv = (torch.empty(k.shape, dtype=k.dtype, device=k.device) for _ in range(2))
        tdp_cross_attn_grad(ctx.plan, q, k, v, mask, out, lse, _dense(dout), dq, dk, dv, scale=ctx.scale)
        return None, dq, dk, dv, None, None


class _DropoutAdd(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, x, res, p, rng):
        x = _dense(x)
        out = torch.empty_like(x)
        tdp_dropout_add(plan, x, None if res is None else _dense(res), p, rng, out)
        ctx.plan, ctx.p, ctx.residual = plan, p, res is not None
        # the gradient draws the same words: it needs this call's seed and offset, not later ones
        ctx.save_for_backward(rng.clone())
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        dout = _dense(dout)
        dx = torch.empty_like(dout)
        tdp_dropout_grad(ctx.plan, dout, ctx.p, ctx.saved_tensors[0], dx)
        return None, dx, dout if ctx.residual else None, None, None


def group_norm(plan: Plan, x, groups, gamma=None, beta=None, eps=1e-5, act="none"):
    """act(group norm of every (tile, item) of tile-major rows x [R, C]) with gradients for x, gamma and beta."""
    return _GroupNorm.apply(plan, x, groups, gamma, beta, eps, act)


def cross_attn(plan: Plan, q, k, v, mask=None, scale=None):
    """Tile rows q [R, Hq, D] attend to states k, v [B, S, Hkv, D] under mask [B, S] or [n_tiles, B, S];
    gradients for q, k and v.  torch sees when it has changed one of them, or the mask, before the gradient, and
    raises an error; it does not see what this library's calls (tdp_norm_filter's keep) write into them."""
    return _CrossAttn.apply(plan, q, k, v, mask, scale)


def dropout_add(plan: Plan, x, res, p, rng):
    """res + dropout(x) with the generator of rng (two 64-bit integers on the device: seed, offset); gradients for
    x and res.  The caller moves the offset on between calls."""
    return _DropoutAdd.apply(plan, x, res, p, rng)


class TileBlock(torch.nn.Module):
    """x + dropout(W_o attn(W_q silu(group_norm(x)), W_kv states)) on tile-major rows x [R, C].

    One plan serves any width: its C is not used by the operators.

    While training with p > 0 each call draws its mask from rng (two 64-bit integers on the device: seed, offset) and
    leaves it as it is.  Blocks, or steps, that are given the same two drop the same elements: move the offset on between any two
    calls, or give each block a seed of its own."""

    def __init__(self, channels, heads, kv_heads, head_dim, context, groups, p=0.0, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        kw = dict(dtype=dtype, device=device)
        self.heads, self.kv_heads, self.head_dim, self.groups, self.p = heads, kv_heads, head_dim, groups, p
        self.gamma = torch.nn.Parameter(torch.ones(channels, **kw))
        self.beta = torch.nn.Parameter(torch.zeros(channels, **kw))
        self.to_q = torch.nn.Linear(channels, heads * head_dim, bias=False, **kw)
        self.to_kv = torch.nn.Linear(context, 2 * kv_heads * head_dim, bias=False, **kw)
        self.to_out = torch.nn.Linear(heads * head_dim, channels, bias=False, **kw)

    def forward(self, plan: Plan, x, states, mask=None, rng=None):
        h = group_norm(plan, x, self.groups, self.gamma, self.beta, act="silu")
        q = self.to_q(h).view(-1, self.heads, self.head_dim)
        kv = self.to_kv(states).view(*states.shape[:2], 2, self.kv_heads, self.head_dim)
        a = self.to_out(cross_attn(plan, q, kv[:, :, 0], kv[:, :, 1], mask).flatten(1))
        return dropout_add(plan, a, x, self.p, rng) if self.training and self.p > 0 else x + a
