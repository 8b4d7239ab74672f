"""Layer norm and the expert exchange under autograd, and an expert block around Fp8Linear.

A pre-norm expert block is

    h  = layer_norm(x)                              # fp8_layernorm_fwd / _bwd
    plan = expert_plan(expert_idx, experts)         # fp8_moe_sort, no gradient
    xs = expert_dispatch(h, plan)                   # fp8_moe_dispatch / _dispatch_bwd
    ys = every expert's linears on its own rows     # Fp8Linear, rows a multiple of 16
    y  = expert_combine(ys, weights, plan)          # fp8_moe_combine / _combine_bwd

Padding rows of xs are zero and so are the gradients of ys there, so an expert's linears run on
padded rows without masks: nothing is added to weight or bias gradients, and without biases (and
with an activation that maps 0 to 0) nothing to amaxes. After a linear with a bias the padding
rows hold the activation of the bias, which the amax of the next linear's input includes.
Everything runs on the current stream; gradients of gradients are not defined.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

from . import _abi
from .autograd import Fp8Linear


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """t as a [rows, cols] tensor that the kernels can read in place, else a copy (an expanded
    or transposed gradient)."""
    t = t.reshape(-1, t.shape[-1])
    r, c = t.shape
    if (c <= 1 or t.stride(1) == 1) and (r <= 1 or t.stride(0) >= c):
        return t
    return t.contiguous()


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, gamma, beta, eps):
        want = x2d.requires_grad or (gamma is not None and gamma.requires_grad)
        y, mean, rstd = _abi.fp8_layernorm_fwd(x2d, gamma, beta, eps=eps, want_stats=want)
        ctx.save_for_backward(x2d, mean, rstd, gamma)
        ctx.beta = None if beta is None else (beta.dtype, beta.shape)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2d, mean, rstd, gamma = ctx.saved_tensors
        want_dx, want_dg, want_db = ctx.needs_input_grad[:3]
        dy = _as_rows(dy)
        if mean is None:                # only beta's gradient, which needs no statistics
            mean = rstd = dy.new_zeros(dy.shape[0], dtype=torch.float32)
        dx, dgamma, dbeta = _abi.fp8_layernorm_bwd(
            dy, x2d, mean, rstd, gamma, want_dx=want_dx, want_dgamma=want_dg,
            want_dbeta=want_db, param_dtype=None if ctx.beta is None else ctx.beta[0])
        return dx, dgamma, dbeta, None


def layer_norm(x, gamma=None, beta=None, eps: float = 1e-5):
    """Layer norm over the last dimension of x (bf16, f16 or f32), differentiable in x, gamma
    and beta. gamma and beta [cols] have x's dtype or float32, both the same."""
    x2d = _as_rows(x)
    return _LayerNormFn.apply(x2d, gamma, beta, eps).reshape(x.shape)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension, with its parameters in ``dtype`` (that of the inputs,
    or float32)."""

    def __init__(self, cols: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype=torch.float32):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(cols, device=device, dtype=dtype))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(cols, device=device, dtype=dtype))
        else:
            self.register_parameter("bias", None)

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)


class ExpertPlan(NamedTuple):
    """Where every (token, choice) pair goes; the index tensors of fp8_moe_sort, on the device."""
    slot: torch.Tensor          # int32 [tokens, topk]: the pair's row, -1: dropped
    source: torch.Tensor        # int32 [rows]: the row's pair, -1: padding
    counts: torch.Tensor        # int32 [experts]
    offsets: torch.Tensor       # int32 [experts + 1]: the experts' first rows


def expert_plan(expert_idx, experts: int, multiple: int = 16) -> ExpertPlan:
    """Sort the pairs of expert_idx [tokens, topk] (int32 or int64, outside [0, experts):
    dropped) by expert, every expert's rows padded to a multiple of ``multiple``."""
    return ExpertPlan(*_abi.fp8_moe_sort(expert_idx, experts, multiple))


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, slot, source):
        ctx.save_for_backward(slot)
        return _abi.fp8_moe_dispatch(x2d, slot, source)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        slot, = ctx.saved_tensors
        return _abi.fp8_moe_dispatch_bwd(_as_rows(dxs), slot), None, None


def expert_dispatch(x, plan: ExpertPlan):
    """x's rows [tokens, cols] in the order of the plan, [rows, cols], 0 in padding rows."""
    return _DispatchFn.apply(_as_rows(x), plan.slot, plan.source)


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, slot, source):
        ctx.save_for_backward(ys, weights, slot, source)
        return _abi.fp8_moe_combine(ys, slot, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weights, slot, source = ctx.saved_tensors
        dys, dw = _abi.fp8_moe_combine_bwd(_as_rows(dy), ys, slot, source, weights)
        need = ctx.needs_input_grad
        return dys if need[0] else None, dw if need[1] else None, None, None


def expert_combine(ys, weights, plan: ExpertPlan):
    """Every token's rows of ys [rows, cols] added with its weights, float32 [tokens, topk]."""
    return _CombineFn.apply(_as_rows(ys), weights.contiguous(), plan.slot, plan.source)


class ExpertBlock(torch.nn.Module):
    """x + experts(layer_norm(x)) of bf16 tokens: a router picks ``topk`` of ``experts``
    two-layer MLPs for each token. The MLPs are Fp8Linear layers, so inside ``fp8_autocast``
    they run in FP8 and outside in bf16. Tokens whose choice is masked (``expert_mask``
    [experts] False) go to the others. The experts' row ranges are read back to the host once
    per forward, since each expert's products are launches of their own."""

    def __init__(self, cols: int, hidden: int, experts: int, topk: int, device=None,
                 eps: float = 1e-5):
        super().__init__()
        if not 1 <= topk <= experts:
            raise ValueError(f"topk={topk} outside [1, {experts}]")
        self.topk, self.experts = topk, experts
        self.norm = LayerNorm(cols, eps, device=device)
        self.router = torch.nn.Linear(cols, experts, bias=False, device=device,
                                      dtype=torch.bfloat16)
        self.up = torch.nn.ModuleList(Fp8Linear(cols, hidden, device=device)
                                      for _ in range(experts))
        self.down = torch.nn.ModuleList(Fp8Linear(hidden, cols, device=device)
                                        for _ in range(experts))

    def route(self, h, expert_mask=None):
        """(expert_idx, weights) of the normed tokens: the topk experts and their softmax."""
        logits = self.router(h).float()
        if expert_mask is not None:
            logits = logits.masked_fill(~expert_mask, float("-inf"))
        top, idx = torch.topk(logits, self.topk, dim=1)
        # a choice without any expert left is dropped; its weight is 0
        gone = torch.isneginf(top)
        weights = torch.softmax(top.masked_fill(gone, -1e30), dim=1).masked_fill(gone, 0.0)
        return idx.masked_fill(gone, -1), weights

    def forward(self, x, expert_mask=None):
        cols = self.norm.weight.shape[0]
        if x.dtype != torch.bfloat16 or x.shape[-1] != cols:
            raise ValueError(f"expected bfloat16 tokens of width {cols}, got {x.dtype} of shape "
                             f"{tuple(x.shape)}")
        x2d = x.reshape(-1, cols)
        h = self.norm(x2d)
        idx, weights = self.route(h, expert_mask)
        plan = expert_plan(idx, self.experts)
        xs = expert_dispatch(h, plan)
        at = plan.offsets.tolist()
        outs = [self.down[e](F.relu(self.up[e](xs[at[e]:at[e + 1]])))
                for e in range(self.experts) if at[e + 1] > at[e]]
        outs.append(xs.new_zeros((xs.shape[0] - at[-1], xs.shape[1])))
        y = expert_combine(torch.cat(outs), weights, plan)
        return (x2d + y).reshape(x.shape)
