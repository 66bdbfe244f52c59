"""Plain float64 forms of the training-step operators (include/q8train.h),
written from their formulas, with gradients by automatic differentiation."""
import math

import torch

RMS, LAYER, NONE = 1, 2, 0


def act(g, kind):
    if kind == 0:
        return g / (1 + torch.exp(-g))
    if kind == 1:
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return 0.5 * g * (1 + torch.erf(g / math.sqrt(2)))


def gated_ff(x, wg, wu, kind):
    return act(x @ wg.T, kind) * (x @ wu.T)


def norm(v, kind, w, b, eps):
    if kind == NONE:
        return v
    if kind == LAYER:
        v = v - v.mean(1, keepdim=True)
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    n = n if w is None else n * w
    return n if b is None else n + b


def block_norm(r, y, post, pre, gate, gate_tokens, scale, eps):
    """post, pre: (kind, weight, bias)."""
    p = norm(y, *post, eps)
    if gate is not None:
        p = p * gate.view(-1, y.shape[1])[torch.arange(y.shape[0], device=y.device) // gate_tokens]
    out = scale * r + p
    return out, norm(out, *pre, eps)


def distill(z, ids, teacher, labels, tau, kd, ce):
    """Row losses, one row at a time."""
    rows = []
    V = z.shape[1]
    for t in range(z.shape[0]):
        row = z.new_zeros(())
        ok = ((ids[t] >= 0) & (ids[t] < V)).nonzero()[:, 0] if ids is not None else []
        if len(ok) and kd > 0 and torch.isfinite(teacher[t][ok]).any():
            logp = torch.log_softmax(teacher[t][ok] / tau, 0)
            keep = torch.isfinite(logp)
            logq = torch.log_softmax(z[t] / tau, 0)[ids[t][ok]]
            row = row + kd * tau ** 2 * (logp.exp()[keep] * (logp - logq)[keep]).sum()
        if labels is not None and ce > 0 and 0 <= int(labels[t]) < V:
            row = row + ce * (torch.logsumexp(z[t], 0) - z[t, int(labels[t])])
        rows.append(row)
    return torch.stack(rows) if rows else z.new_zeros(0)
