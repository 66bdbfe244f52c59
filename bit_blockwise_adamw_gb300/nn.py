"""Autograd functions and modules over the training-step operators
(include/q8train.h): what comes before the optimizers of
bit_blockwise_adamw_gb300.optim in a step.

All of them run on CUDA in bf16 (the norms' residual stream, the embedding's
output and the loss's logits also in float32), on the current stream, and accept
any leading dimensions.  A module's parameters are contiguous bf16 tensors, as the
optimizers want them.
"""
import torch
from torch import nn
import torch.nn.functional as F

from . import _binding as B

ACTIVATIONS = {"silu": B.SILU, "gelu_tanh": B.GELU_TANH, "gelu": B.GELU}
NORMS = {None: B.NORM_NONE, "none": B.NORM_NONE, "rms": B.NORM_RMS, "layer": B.NORM_LAYER}


def _flat(t):
    """t as a matrix the operators take: rows of unit stride that do not overlap."""
    t = t.reshape(t.shape[:-1].numel(), t.shape[-1])
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] else t.contiguous()


class _GatedFF(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act, keep):
        h = torch.empty(x.shape[0], w_gate.shape[0], dtype=x.dtype, device=x.device)
        saved = None
        if keep and any(ctx.needs_input_grad[:3]):
            saved = torch.empty(2, *h.shape, dtype=torch.float32, device=x.device)
        B.q8_gated_ff_forward(x, w_gate, w_up, h, act, saved=saved)
        ctx.save_for_backward(x, w_gate, w_up, saved)
        ctx.act = act
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, w_gate, w_up, saved = ctx.saved_tensors
        out = [torch.empty(t.shape, dtype=t.dtype, device=t.device) if need else None
               for t, need in zip((x, w_gate, w_up), ctx.needs_input_grad)]
        B.q8_gated_ff_backward(x, w_gate, w_up, dh.contiguous(), *out, ctx.act, saved=saved)
        return (*out, None, None)


def gated_ff(x, w_gate, w_up, activation="silu", recompute=False):
    """act(x w_gate^T) * (x w_up^T), differentiable in all three.  Both
    projections are kept in float32 for the backward pass; recompute=True keeps
    nothing and computes them again there."""
    keep = not recompute and torch.is_grad_enabled()     # needs_input_grad is true of a parameter under no_grad, too
    return _GatedFF.apply(_flat(x), w_gate, w_up, ACTIVATIONS[activation], keep).view(*x.shape[:-1], w_gate.shape[0])


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, y, post_weight, post_bias, pre_weight, pre_bias, gate, kinds, scale, eps, gate_tokens):
        out = torch.empty(residual.shape, dtype=residual.dtype, device=residual.device)
        z = torch.empty(y.shape, dtype=y.dtype, device=y.device)
        ctx.kw = dict(post_weight=post_weight, post_bias=post_bias, pre_weight=pre_weight, pre_bias=pre_bias, gate=gate)
        ctx.opts = dict(residual_scale=scale, eps=eps, gate_tokens=gate_tokens)
        ctx.kinds = kinds
        B.q8_block_norm_forward(residual, y, out, z, *kinds, **ctx.kw, **ctx.opts)
        ctx.save_for_backward(residual, y, *ctx.kw.values())
        ctx.kw = None
        ctx.set_materialize_grads(False)
        return out, z

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out, dz):
        residual, y, *vectors = ctx.saved_tensors
        names = ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")
        tensors = (residual, y, *vectors)
        grads = [torch.empty(t.shape, dtype=t.dtype, device=t.device) if need and t is not None else None
                 for t, need in zip(tensors, ctx.needs_input_grad)]
        B.q8_block_norm_backward(residual, y, None if d_out is None else d_out.contiguous(),
                                 None if dz is None else dz.contiguous(), grads[0], grads[1], *ctx.kinds,
                                 **dict(zip(names, vectors)), **ctx.opts,
                                 **{"d" + n: g for n, g in zip(names, grads[2:])})
        return (*grads, None, None, None, None)


def block_norm(residual, y, post="rms", pre="rms", post_weight=None, post_bias=None, pre_weight=None, pre_bias=None,
               gate=None, residual_scale=1.0, eps=1e-5):
    """(r', z): r' = residual_scale * residual + gate * N_post(y), z = N_pre(r').
    gate: [dim], or a row for each group of consecutive tokens [groups, dim]."""
    shape = y.shape
    groups = 1 if gate is None or gate.dim() == 1 else gate.shape[0]
    tokens = y.numel() // shape[-1]
    if tokens % groups:
        raise ValueError("gate's rows must divide the tokens")
    out, z = _BlockNorm.apply(_flat(residual), _flat(y), post_weight, post_bias, pre_weight, pre_bias, gate,
                              (NORMS[post], NORMS[pre]), float(residual_scale), float(eps), max(1, tokens // groups))
    return out.view(shape), z.view(shape)


class _DistillTopK(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, labels, temperature, kd_weight, ce_weight, keep):
        rows = logits.shape[0]
        loss = torch.empty(rows, dtype=torch.float32, device=logits.device)
        stats = torch.empty(rows, 2, dtype=torch.float32, device=logits.device) if keep and ctx.needs_input_grad[0] else None
        ctx.opts = dict(temperature=temperature, kd_weight=kd_weight, ce_weight=ce_weight)
        B.q8_distill_topk_forward(logits, ids, teacher, loss, stats=stats, labels=labels, **ctx.opts)
        ctx.save_for_backward(logits, ids, teacher, labels, stats)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        logits, ids, teacher, labels, stats = ctx.saved_tensors
        d = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        B.q8_distill_topk_backward(logits, ids, teacher, stats, d, labels=labels, row_weight=dloss.float().contiguous(),
                                   **ctx.opts)
        return d, None, None, None, None, None, None, None


def distill_topk(logits, teacher_ids, teacher_logits, labels=None, temperature=1.0, kd_weight=1.0, ce_weight=0.0):
    """Each row's distillation loss in float32 (q8_distill_topk_forward): the
    teacher's top entries as torch.topk gives them (ids outside the vocabulary
    are padding), labels outside it (-100) are not counted.  Without a teacher
    (None for both) the labels' term is left.  Differentiable in the logits."""
    if (teacher_ids is None) != (teacher_logits is None):
        raise ValueError("teacher_ids and teacher_logits go together")
    rows = logits.shape[:-1]
    ids, teacher = (None, None) if teacher_ids is None else \
        (_flat(teacher_ids).contiguous(), _flat(teacher_logits).float().contiguous())
    loss = _DistillTopK.apply(_flat(logits), ids, teacher, None if labels is None else labels.reshape(-1).contiguous(),
                              float(temperature), float(kd_weight), float(ce_weight), torch.is_grad_enabled())
    return loss.view(rows)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, dtype):
        out = torch.empty(ids.shape[0], weight.shape[1], dtype=dtype, device=weight.device)
        B.q8_embedding_forward(ids, weight, out, scale)
        ctx.save_for_backward(ids)
        ctx.shape, ctx.scale = weight.shape, scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        dw = torch.empty(ctx.shape, dtype=torch.bfloat16, device=dout.device)
        B.q8_embedding_backward(ids, _flat(dout), dw, ctx.scale)
        return None, dw, None, None


def embedding(ids, weight, scale=1.0, dtype=torch.bfloat16):
    """scale * weight[ids] in bf16 or float32, differentiable in weight: ids
    outside the table (-100 and the like) are no tokens, their rows are zeros.
    The same ids and gradients give the same bits."""
    return _Embedding.apply(ids.reshape(-1).contiguous(), weight, float(scale), dtype).view(*ids.shape, weight.shape[1])


class Embedding(nn.Module):
    """The token embedding, its rows scaled (by the root of the width, where a
    model does so)."""

    def __init__(self, vocab, dim, scale=1.0, dtype=torch.bfloat16, std=0.02, device=None):
        super().__init__()
        self.weight = nn.Parameter(torch.empty(vocab, dim, dtype=torch.bfloat16, device=device))
        self.scale, self.dtype = scale, dtype
        nn.init.normal_(self.weight, std=std)

    def forward(self, ids):
        return embedding(ids, self.weight, self.scale, self.dtype)


class GatedFeedForward(nn.Module):
    """down(act(gate(x)) * up(x)) without biases."""

    def __init__(self, d_model, d_ff, activation="silu", recompute=False, device=None):
        super().__init__()
        kw = dict(dtype=torch.bfloat16, device=device)
        self.w_gate = nn.Parameter(torch.empty(d_ff, d_model, **kw))
        self.w_up = nn.Parameter(torch.empty(d_ff, d_model, **kw))
        self.w_down = nn.Parameter(torch.empty(d_model, d_ff, **kw))
        self.activation, self.recompute = activation, recompute
        for w in self.parameters():
            nn.init.normal_(w, std=w.shape[1] ** -0.5)

    def forward(self, x):
        return F.linear(gated_ff(x, self.w_gate, self.w_up, self.activation, self.recompute), self.w_down)


class BlockNorm(nn.Module):
    """The norm after a block and the one before the next, with a learned
    channel gate: forward(residual, y) -> (residual', z)."""

    def __init__(self, dim, post="rms", pre="rms", gate=True, residual_scale=1.0, eps=1e-5, device=None):
        super().__init__()
        kw = dict(dtype=torch.bfloat16, device=device)
        self.post, self.pre, self.residual_scale, self.eps = post, pre, residual_scale, eps
        for name, kind in (("post", post), ("pre", pre)):
            weight = nn.Parameter(torch.ones(dim, **kw)) if NORMS[kind] != B.NORM_NONE else None
            bias = nn.Parameter(torch.zeros(dim, **kw)) if NORMS[kind] == B.NORM_LAYER else None
            self.register_parameter(name + "_weight", weight)
            self.register_parameter(name + "_bias", bias)
        self.register_parameter("gate", nn.Parameter(torch.ones(dim, **kw)) if gate else None)

    def forward(self, residual, y):
        return block_norm(residual, y, self.post, self.pre, self.post_weight, self.post_bias, self.pre_weight,
                          self.pre_bias, self.gate, self.residual_scale, self.eps)
