"""Layer norm, router, expert exchange and experts under autograd, and two expert blocks.

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

With the router and the experts' products of the block recipe nothing is read back to the host:

    r  = expert_route(logits, topk)                 # fp8_moe_route / _bwd, with both losses
    plan = expert_plan(r.expert_idx, experts, 128)
    ys = expert_mlp(xs, w_up, w_down, plan)         # fp8_grouped_linear_*, fp8_act_quantize / _bwd

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
    # a copy also where an expanded tensor without elements calls itself contiguous
    return t.contiguous() if r * c else t.clone(memory_format=torch.contiguous_format)


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


class _PlanTensors(NamedTuple):
    slot: torch.Tensor          # int32 [tokens, topk]: the pair's row, -1: dropped
    source: torch.Tensor        # int32 [rows]: the row's pair, -1: padding
    counts: torch.Tensor        # int32 [experts]
    offsets: torch.Tensor       # int32 [experts + 1]: the experts' first rows


class ExpertPlan(_PlanTensors):
    """Where every (token, choice) pair goes; the four index tensors of fp8_moe_sort, on the device.
    ``multiple`` is what the plan was made with, None for a plan made of the tensors alone."""
    multiple = None


def expert_plan(expert_idx, experts: int, multiple: int = 16) -> ExpertPlan:
    """Sort the pairs of expert_idx [tokens, topk] (int32 or int64, outside [0, experts):
    dropped) by expert, every expert's rows padded to a multiple of ``multiple``."""
    plan = ExpertPlan(*_abi.fp8_moe_sort(expert_idx, experts, multiple))
    plan.multiple = multiple
    return plan


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


class Routing(NamedTuple):
    """What expert_route gives. expert_idx and counts have no gradient."""
    expert_idx: torch.Tensor    # int32 [tokens, topk], -1: no expert
    weights: torch.Tensor       # float32 [tokens, topk]
    counts: torch.Tensor        # int32 [experts]: the pairs that chose the expert
    balance_loss: torch.Tensor  # float32: 1 where the experts are evenly used
    z_loss: torch.Tensor        # float32: mean of the squared log-sum-exp


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, normalize, tokens_valid):
        idx, w, lse, counts, losses = _abi.fp8_moe_route(logits, topk, tokens_valid, normalize)
        ctx.save_for_backward(logits, lse, idx, w, counts)
        ctx.args = (tokens_valid, normalize)
        ctx.mark_non_differentiable(idx, counts)
        ctx.set_materialize_grads(False)
        return idx, w, counts, losses

    @staticmethod
    @once_differentiable
    def backward(ctx, _idx, dw, _counts, dlosses):
        logits, lse, idx, w, counts = ctx.saved_tensors
        tokens_valid, normalize = ctx.args
        return _abi.fp8_moe_route_bwd(
            logits, lse, idx, w, counts, None if dw is None else dw.contiguous(),
            None if dlosses is None else dlosses.contiguous(), tokens_valid, normalize), \
            None, None, None


def expert_route(logits, topk: int, normalize: bool = True, tokens_valid=None) -> Routing:
    """The topk experts of each token of logits [tokens, experts] (bf16, f16 or f32) and their
    weights, with the losses that keep the experts evenly used; see fp8_moe_route."""
    idx, w, counts, losses = _RouteFn.apply(_as_rows(logits), topk, normalize, tokens_valid)
    return Routing(idx, w, counts, losses[0], losses[1])


def _quantize_rows(x, transposed: bool):
    """(q, scale, q_t, scale_t) in 1x128 tiles."""
    q, q_t, _, scale, scale_t = _abi.fp8_quantize_amax(
        x, gran=_abi.FP8_BLOCK_1x128, want_q_t=transposed, want_amax=False)
    return q, scale, q_t, scale_t


# The products take weights whose rows are fewer codes than this apart.
_ROW_STRIDE_LIMIT = 1 << 23


def _quantize_experts(w, transposed: bool):
    """Stacked weights [experts, n, k] in 128x128 tiles: codes and scales [experts, n, k], and
    transposed as [experts, k, n]. The transposed rows of all experts alternate in memory; a stack
    whose rows would be too far apart for the products is copied expert by expert."""
    e, n, k = w.shape
    q, q_t, _, scale, scale_t = _abi.fp8_quantize_amax(
        w.reshape(e * n, k), gran=_abi.FP8_BLOCK_128x128, want_q_t=transposed, want_amax=False)
    first = (q.view(e, n, k), scale.view(e, n // 128, k // 128))
    if not transposed:
        return first, (None, None)
    q_t = q_t.view(k, e, n).transpose(0, 1)
    if e * n >= _ROW_STRIDE_LIMIT:
        q_t = q_t.contiguous()
    return first, (q_t, scale_t.view(k // 128, e, n // 128).transpose(0, 1))


class _ExpertMlpFn(torch.autograd.Function):
    """Kept between the passes: the transposed codes of x, a and the weights, and h in 8 bits; for
    a gated h 3 bytes an element of a, against 5 with h in bf16."""

    @staticmethod
    def forward(ctx, xs, w_up, w_down, offsets, counts, act, gated, max_rows, grad):
        # `grad`: whether the graph is recorded, which needs_input_grad does not tell
        want_x, want_up, want_down = (grad and need for need in ctx.needs_input_grad[:3])
        want_h = want_x or want_up
        qx, sx, qx_t, sx_t = _quantize_rows(xs, want_up)
        (q1, s1), up_t = _quantize_experts(w_up, want_x)
        h = _abi.fp8_grouped_linear_fwd(qx, q1, sx, s1, offsets, counts, max_rows=max_rows)
        qa, sa, qa_t, sa_t, hq, hs = _abi.fp8_act_quantize(h, act, gated, want_q_t=want_down,
                                                           want_checkpoint=want_h)
        del h
        (q2, s2), down_t = _quantize_experts(w_down, want_h)
        ys = _abi.fp8_grouped_linear_fwd(qa, q2, sa, s2, offsets, counts, max_rows=max_rows)
        ctx.save_for_backward(qx_t, sx_t, *up_t, qa_t, sa_t, hq, hs, *down_t, offsets, counts)
        ctx.args = (act, gated, max_rows)
        return ys

    @staticmethod
    @once_differentiable
    def backward(ctx, dys):
        qx_t, sx_t, q1_t, s1_t, qa_t, sa_t, hq, hs, q2_t, s2_t, offsets, counts = ctx.saved_tensors
        act, gated, max_rows = ctx.args
        want_x, want_up, want_down = ctx.needs_input_grad[:3]
        qg, sg, qg_t, sg_t = _quantize_rows(dys.contiguous(), want_down)
        dx = dup = ddown = None
        if want_down:
            ddown = _abi.fp8_grouped_linear_wgrad(qg_t, qa_t, sg_t, sa_t, offsets, counts)
        if want_x or want_up:
            da = _abi.fp8_grouped_linear_dgrad(qg, q2_t, sg, s2_t, offsets, counts,
                                               max_rows=max_rows)
            qh, sh, qh_t, sh_t, _ = _abi.fp8_act_quantize_bwd(da, hq, hs, act, gated,
                                                              want_q=want_x, want_q_t=want_up)
            if want_up:
                dup = _abi.fp8_grouped_linear_wgrad(qh_t, qx_t, sh_t, sx_t, offsets, counts)
            if want_x:
                dx = _abi.fp8_grouped_linear_dgrad(qh, q1_t, sh, s1_t, offsets, counts,
                                                   max_rows=max_rows)
        return dx, dup, ddown, None, None, None, None, None, None


def _check_whole_blocks(plan: ExpertPlan, weight_grads: bool):
    """Refuse a plan whose experts do not begin at multiples of 128 rows. The row count cannot tell
    (200 pairs of 2 experts take 384 rows with multiple 96 and with 128), so without the plan's
    multiple the offsets are read back, if weights have gradients: only those take whole blocks."""
    if plan.multiple is not None:
        whole = plan.multiple % 128 == 0
    elif not weight_grads:
        return
    elif plan.offsets.is_cuda and torch.cuda.is_current_stream_capturing():
        raise ValueError("the offsets of a plan that expert_plan did not make cannot be read back "
                         "during a capture")
    else:
        whole = not (plan.offsets % 128).any().item()
    if not whole:
        raise ValueError("an expert of the plan does not begin at a multiple of 128 rows: blocks of "
                         "128 rows would mix experts (expert_plan with multiple=128)")


def expert_mlp(xs, w_up, w_down, plan: ExpertPlan, act: str = "silu", gated: bool = True):
    """Every expert's two linears with the activation between them, on its rows of xs [rows, cols]
    (bf16, sorted by a plan with multiple 128), by the block recipe and without reading the row
    counts back: act(xs W_up^T) W_down^T, or with ``gated`` act(g) u of [g | u] = xs W_up^T. w_up
    [experts, hidden or 2 hidden, cols] and w_down [experts, cols, hidden] are bf16, cols and hidden
    multiples of 128. Rows of no expert give 0. For the backward the activation's input is kept in 8
    bits. The gradient of ys has to be finite in padding rows (expert_combine's is 0 there). Where a
    weight has a gradient, the offsets of a plan that expert_plan did not make are read back to check
    that they are multiples of 128."""
    xs = _as_rows(xs)
    e, cols, hidden = w_down.shape
    width = 2 * hidden if gated else hidden
    if tuple(w_up.shape) != (e, width, cols):
        raise ValueError(f"w_up has shape {tuple(w_up.shape)}, expected {(e, width, cols)}")
    if plan.counts.numel() != e:
        raise ValueError(f"the plan is for {plan.counts.numel()} experts, the weights for {e}")
    if cols % 128 or hidden % 128:
        raise ValueError(f"cols={cols} and hidden={hidden} must be multiples of 128")
    if xs.shape[0] % 128 or xs.shape[0] != plan.source.numel():
        raise ValueError(f"xs has {xs.shape[0]} rows, the plan {plan.source.numel()}; both have to "
                         "be the same multiple of 128 (expert_plan with multiple=128)")
    for t, name in ((xs, "xs"), (w_up, "w_up"), (w_down, "w_down")):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    least = _abi.fp8_moe_rows(*plan.slot.shape, e, 128)
    if xs.shape[0] < least:         # of another multiple: blocks of 128 rows would mix experts
        raise ValueError(f"the plan has {xs.shape[0]} rows, with multiple=128 it has {least}")
    grad = torch.is_grad_enabled()
    _check_whole_blocks(plan, grad and (w_up.requires_grad or w_down.requires_grad))
    return _ExpertMlpFn.apply(xs.contiguous(), w_up, w_down, plan.offsets, plan.counts, act, gated,
                              plan.slot.shape[0], grad)


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


class GroupedExpertBlock(torch.nn.Module):
    """x + experts(layer_norm(x)) of bf16 tokens, all experts at once: a router picks ``topk`` of
    ``experts`` MLPs (gated SiLU by default) for each token, and their products run by the block
    recipe over the sorted tokens, without reading anything back to the host. ``forward`` returns the
    tokens and the Routing, whose losses are to be added to the training loss. cols and hidden must be
    multiples of 128."""

    def __init__(self, cols: int, hidden: int, experts: int, topk: int, device=None,
                 eps: float = 1e-5, act: str = "silu", gated: bool = True):
        super().__init__()
        if not 1 <= topk <= experts:
            raise ValueError(f"topk={topk} outside [1, {experts}]")
        if cols % 128 or hidden % 128:
            raise ValueError(f"cols={cols} and hidden={hidden} must be multiples of 128")
        self.topk, self.experts, self.act, self.gated = topk, experts, act, gated
        self.norm = LayerNorm(cols, eps, device=device)
        bf16 = dict(device=device, dtype=torch.bfloat16)
        self.router = torch.nn.Linear(cols, experts, bias=False, **bf16)
        self.w_up = torch.nn.Parameter(
            torch.empty((experts, 2 * hidden if gated else hidden, cols), **bf16))
        self.w_down = torch.nn.Parameter(torch.empty((experts, cols, hidden), **bf16))
        for w in (self.w_up, self.w_down):          # as nn.Linear's default
            bound = 1.0 / w.shape[2] ** 0.5
            torch.nn.init.uniform_(w, -bound, bound)

    def forward(self, x, expert_mask=None):
        cols = self.norm.weight.shape[0]
        if x.dtype != torch.bfloat16 or x.shape[-1] != cols:
            raise ValueError(f"expected bfloat16 tokens of width {cols}, got {x.dtype} of shape "
                             f"{tuple(x.shape)}")
        x2d = x.reshape(-1, cols)
        h = self.norm(x2d)
        logits = self.router(h).float()
        if expert_mask is not None:
            logits = logits.masked_fill(~expert_mask, float("-inf"))
        r = expert_route(logits, self.topk)
        plan = expert_plan(r.expert_idx, self.experts, 128)
        ys = expert_mlp(expert_dispatch(h, plan), self.w_up, self.w_down, plan, self.act, self.gated)
        return (x2d + expert_combine(ys, r.weights, plan)).reshape(x.shape), r
