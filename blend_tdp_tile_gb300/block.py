"""The per-tile block's operators as differentiable torch functions, and a block made of them.

Between ``tdp_split`` and ``tdp_blend`` a transformer runs on every tile.  The functions here
put the library's operators on tile-major rows under torch's autograd:

  group_norm(plan, x, groups, gamma, beta)   statistics of every (tile, item), channels last, SiLU
  cross_attn(plan, q, k, v, mask)            tile rows attend to an encoder's states
  dropout_add(plan, x, res, p, rng)          residual + dropout whose mask is never stored
  rms_norm(plan, x, w, res)                  residual + root-mean-square norm; its checkpoint in 8 bits, if asked for
  rope(plan, x, Q, table)                    heads turned by the positions that the split hands out

``TileBlock`` is one cross-attention sublayer of them: normalise, project, attend, project back,
drop out and add.  ``RotaryBlock`` attends to the conditioning tokens that each tile keeps, at their positions, and serves
with its projections in 8 bits (``Linear8``).  All tiles go through each call at once; nothing is padded.  The gradients are first ones: a
derivative of theirs raises an error.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (Plan, tdp_cross_attn, tdp_cross_attn_grad, tdp_dropout_add, tdp_dropout_grad, tdp_group_norm,
               tdp_group_norm_grad, tdp_matmul8, tdp_quant8, tdp_rms_norm, tdp_rms_norm_grad, tdp_rope, tdp_rope_freqs,
               tdp_rope_grad, tdp_rope_table)

__all__ = ["group_norm", "cross_attn", "dropout_add", "rms_norm", "rope", "quant8", "Linear8", "TileBlock", "RotaryBlock"]


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


def _heads(t):
    """t [rows, heads, D] as tdp_rope takes it: strides and start on 16 bytes."""
    unit = 16 // t.element_size()
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s % unit == 0 for s, n in zip(t.stride()[:2], t.shape) if n > 1)
    return t if ok else _dense(t)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, x, w, res, eps, keep8):
        x, w = _dense(x), None if w is None else _dense(w)
        rows = x.numel() // x.shape[-1]
        y, rstd = torch.empty_like(x), torch.empty(rows, dtype=torch.float32, device=x.device)
        h, res = (x, None) if res is None else (torch.empty_like(x), _dense(res))
        x8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device) if keep8 else None
        scale = torch.empty_like(rstd) if keep8 else None
        tdp_rms_norm(plan, x, w, y, res=res, h=None if res is None else h, rstd=rstd, x8=x8, x8_scale=scale, eps=eps)
        ctx.plan, ctx.residual = plan, res is not None
        ctx.save_for_backward(w, rstd, None if keep8 else h, x8, scale)
        ctx.set_materialize_grads(False)
        return (y, h) if res is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        w, rstd, h, x8, scale = ctx.saved_tensors
        kept = h if x8 is None else x8
        if dy is None:              # the norm's output has no part in it
            dx = None if dh is None else _dense(dh)
            return None, dx, None, dx if ctx.residual else None, None, None
        dy = _dense(dy)
        dx = torch.empty_like(dy)
        dw = torch.empty(dy.shape[-1], dtype=torch.float32, device=dy.device) if ctx.needs_input_grad[2] else None
        tdp_rms_norm_grad(ctx.plan, dy, dx, w, rstd, h=None if x8 is not None else kept, x8=x8, x8_scale=scale,
                          dh=None if dh is None else _dense(dh), dw=dw)
        return None, dx, None if dw is None else dw.to(w.dtype), dx if ctx.residual else None, None, None


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, x, Q, table, layout, at, scale):
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        tdp_rope(plan, _heads(x), Q, table, out, layout=layout, at=at, scale=scale)
        ctx.plan, ctx.how = plan, dict(layout=layout, at=at, scale=scale)
        ctx.save_for_backward(Q, table)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        Q, table = ctx.saved_tensors
        dx = torch.empty(dout.shape, dtype=dout.dtype, device=dout.device)
        tdp_rope_grad(ctx.plan, _heads(dout), Q, table, dx, **ctx.how)
        return None, dx, None, None, None, None, None


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


def rms_norm(plan: Plan, x, w=None, res=None, eps=1e-6, keep8=False):
    """Root-mean-square norm of the rows of x [.., C], times w [C]; with res, (the norm of x + res, x + res).  Gradients for x, w
    and res.  keep8: what is kept for them is the normalised rows in 8 bits, a quarter of fp32's and half of bf16's bytes,
    and the gradients are of those rows."""
    return _RmsNorm.apply(plan, x, w, res, eps, keep8)


def rope(plan: Plan, x, Q, table, layout="half", at="middle", scale=1.0):
    """Tile rows x [R, heads, D], every head turned by the rows' positions Q (from tdp_split; table from tdp_rope_table);
    gradient for x."""
    return _Rope.apply(plan, x, Q, table, layout, at, float(scale))      # the gradient's too, whatever held it becomes


def quant8(plan: Plan, x):
    """(x8, scale): the rows of x [.., C] in 8 bits.  No gradient."""
    x = _dense(x.detach())
    x8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty(x.numel() // x.shape[-1], dtype=torch.float32, device=x.device)
    tdp_quant8(plan, x, x8, scale)
    return x8, scale


class Linear8(torch.nn.Module):
    """A linear layer with its weights in 8 bits, a scale an output channel, for serving: it has no gradients and raises an
    error where one is asked for.  A change of the module's dtype leaves it alone."""

    def __init__(self, plan: Plan, linear: torch.nn.Linear):
        super().__init__()
        w8, scale = quant8(plan, linear.weight)
        self.register_buffer("w8", w8.view(torch.uint8))
        self.register_buffer("scale", scale)
        self.register_buffer("bias", None if linear.bias is None else linear.bias.detach().clone())

    def _apply(self, fn, recurse=True):
        """Moves what the layer holds; a change of dtype sees bytes, and leaves weights, scales and bias as they are."""
        kept = {n: b.dtype for n, b in self._buffers.items() if b is not None}
        for n in kept:
            self._buffers[n] = self._buffers[n].view(torch.uint8)
        try:
            return super()._apply(fn, recurse)
        finally:
            for n, dtype in kept.items():
                self._buffers[n] = self._buffers[n].view(dtype)

    def forward(self, plan: Plan, x, scale=None, res=None):
        """x [.., K] in the plan's dtype, or in 8 bits with its scale; res: what the product is added to, or None."""
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, res)):
            raise RuntimeError("Linear8 has no gradient: call it under torch.no_grad()")
        x8, scale = quant8(plan, x) if scale is None else (x, scale)
        out = torch.empty((*x8.shape[:-1], self.w8.shape[0]), dtype=plan_dtype(plan), device=x8.device)
        tdp_matmul8(plan, x8, scale, self.w8, self.scale, out, bias=self.bias, res=None if res is None else _dense(res))
        return out


def plan_dtype(plan: Plan):
    """torch's name of the plan's element type."""
    return torch.float32 if plan.esize == 4 else torch.bfloat16


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


class RotaryBlock(torch.nn.Module):
    """x + dropout(W_o attn(rope(W_q rms_norm(x)), rope(W_k tokens), W_v tokens)) on tile-major rows x [R, C]: every tile's rows attend
    to the conditioning tokens that the tile keeps, both turned by their positions.

    pairs: pairs of a head on each of the three axes.  keep8: training keeps the normalised rows in 8 bits.  After to_8bit() the block
    runs its projections in 8 bits, without gradients, until train() brings the full ones back; weights that change in between
    need another to_8bit().  rng as for TileBlock."""

    def __init__(self, channels, heads, kv_heads, head_dim, context, pairs, p=0.0, keep8=False, base=10000.0, scaling="none", factor=1.0,
                 length=1.0, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        kw = dict(dtype=dtype, device=device)
        self.heads, self.kv_heads, self.head_dim, self.p, self.keep8 = heads, kv_heads, head_dim, p, keep8
        freq, axis, self.scale = tdp_rope_freqs(pairs, base, scaling, factor, length)
        self.register_buffer("table", tdp_rope_table(freq, axis).to(device))
        self.w = torch.nn.Parameter(torch.ones(channels, **kw))
        self.to_q = torch.nn.Linear(channels, heads * head_dim, bias=False, **kw)
        self.to_kv = torch.nn.Linear(context, 2 * kv_heads * head_dim, bias=False, **kw)
        self.to_out = torch.nn.Linear(heads * head_dim, channels, bias=False, **kw)
        self.in8 = None

    def to_8bit(self, plan: Plan):
        self.eval()
        self.in8 = torch.nn.ModuleDict({n: Linear8(plan, getattr(self, n)) for n in ("to_q", "to_kv", "to_out")})
        return self

    def train(self, mode=True):
        if mode:
            self.in8 = None
        return super().train(mode)

    def _load_from_state_dict(self, state_dict, prefix, *args):
        # a served block's state has its projections in 8 bits too: a block without them takes the weights
        if self.in8 is None:
            state_dict = {k: v for k, v in state_dict.items() if not k.startswith(prefix + "in8.")}
        super()._load_from_state_dict(state_dict, prefix, *args)

    def forward(self, plan: Plan, x, Q, tokens_plan: Plan, tokens, P, mask=None, rng=None):
        """Q: tile-major positions of the rows, from tdp_split with normalize = 0, on the tokens' origin.  tokens [B, S, context] at
        P [B, 3, S, 2], with tokens_plan an untiled plan of B items of S tokens.  mask [B, S] or [n_tiles, B, S] (tdp_norm_filter's
        keep), or None."""
        q, kv = (self._project8 if self.in8 is not None else self._project)(plan, x, tokens)
        B, S = tokens.shape[:2]
        kv = kv.view(B * S, 2, self.kv_heads, self.head_dim)
        q = rope(plan, q.view(-1, self.heads, self.head_dim), Q, self.table, scale=self.scale)
        k = rope(tokens_plan, kv[:, 0], P, self.table, scale=self.scale)
        a = cross_attn(plan, q, k.view(B, S, self.kv_heads, self.head_dim), kv.view(B, S, 2, self.kv_heads, self.head_dim)[:, :, 1], mask).flatten(1)
        if self.in8 is not None:
            return self.in8["to_out"](plan, a, res=x)
        a = self.to_out(a)
        return dropout_add(plan, a, x, self.p, rng) if self.training and self.p > 0 else x + a

    def _project(self, plan, x, tokens):
        return self.to_q(rms_norm(plan, x, self.w, keep8=self.keep8)), self.to_kv(tokens)

    def _project8(self, plan, x, tokens):
        if torch.is_grad_enabled() and (x.requires_grad or tokens.requires_grad):
            raise RuntimeError("a block in 8 bits has no gradient: call it under torch.no_grad()")
        x = _dense(x.detach())
        y8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        tdp_rms_norm(plan, x, self.w.detach(), None, y8=y8, y8_scale=scale)
        return self.in8["to_q"](plan, y8, scale), self.in8["to_kv"](plan, tokens)
