"""The autograd functions over the training-step operators without a GPU: what
they pass on and allocate, with the library's calls replaced by recorders."""
import pytest
import torch

from bit_blockwise_adamw_gb300 import nn as q8nn

BF = torch.bfloat16


class Calls:
    """Stands for the binding's functions; keeps each call's arguments."""

    def __init__(self, monkeypatch):
        self.made = []
        for name in ("q8_gated_ff_forward", "q8_gated_ff_backward", "q8_block_norm_forward", "q8_block_norm_backward",
                     "q8_distill_topk_forward", "q8_distill_topk_backward"):
            monkeypatch.setattr(q8nn.B, name, lambda *a, _name=name, **kw: self.made.append((_name, a, kw)))

    def last(self, name):
        return [(a, kw) for n, a, kw in self.made if n == name][-1]


@pytest.fixture
def calls(monkeypatch):
    return Calls(monkeypatch)


@pytest.mark.parametrize("shape", [(0, 8), (3, 0, 8), (0, 5, 8)])
def test_gated_ff_without_tokens(calls, shape):
    x, w = torch.zeros(shape, dtype=BF, requires_grad=True), torch.zeros(24, 8, dtype=BF, requires_grad=True)
    h = q8nn.gated_ff(x, w, w)
    assert h.shape == (*shape[:-1], 24)
    h.sum().backward()
    assert calls.last("q8_gated_ff_backward") and x.grad.shape == x.shape and w.grad.shape == w.shape


@pytest.mark.parametrize("teacher", ["none", "empty"])
@pytest.mark.parametrize("lead", [(4,), (2, 3), ()])
def test_distill_without_teacher_entries(calls, teacher, lead):
    """The labels' term alone: no teacher, or one of no entries."""
    logits = torch.zeros(*lead, 9, requires_grad=True)
    ids, t = (None, None) if teacher == "none" else (torch.zeros(*lead, 0, dtype=torch.int64), torch.zeros(*lead, 0))
    loss = q8nn.distill_topk(logits, ids, t, labels=torch.zeros(lead, dtype=torch.int64), ce_weight=1.0)
    assert loss.shape == lead
    loss.sum().backward()
    rows = logits.numel() // 9
    for name in ("q8_distill_topk_forward", "q8_distill_topk_backward"):
        a, kw = calls.last(name)
        assert a[0].shape == (rows, 9) and kw["labels"].shape == (rows,)
        assert (a[1] is None and a[2] is None) if teacher == "none" else a[1].shape == a[2].shape == (rows, 0)


def test_distill_wants_both_of_the_teacher_or_neither(calls):
    logits = torch.zeros(4, 9)
    for ids, t in ((torch.zeros(4, 2, dtype=torch.int64), None), (None, torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="teacher"):
            q8nn.distill_topk(logits, ids, t)
    assert not calls.made


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_where_no_gradient_follows(calls, mode):
    """Evaluation of a model whose parameters want gradients: no projections in
    float32 beside h, no statistics beside the losses."""
    m = q8nn.GatedFeedForward(8, 24)
    logits = torch.zeros(4, 9, requires_grad=True)
    with mode():
        m(torch.zeros(3, 8, dtype=BF))
        q8nn.distill_topk(logits, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    assert calls.last("q8_gated_ff_forward")[1]["saved"] is None
    assert calls.last("q8_distill_topk_forward")[1]["stats"] is None


def test_what_a_backward_pass_needs_is_kept(calls):
    m = q8nn.GatedFeedForward(8, 24)
    m(torch.zeros(3, 8, dtype=BF))
    assert calls.last("q8_gated_ff_forward")[1]["saved"].shape == (2, 3, 24)
    q8nn.distill_topk(torch.zeros(4, 9, requires_grad=True), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    assert calls.last("q8_distill_topk_forward")[1]["stats"].shape == (4, 2)
    for kw in (dict(recompute=True), dict()):
        q8nn.gated_ff(torch.zeros(3, 8, dtype=BF, requires_grad=bool(kw)), m.w_gate.detach(), m.w_up.detach(), **kw)
        assert calls.last("q8_gated_ff_forward")[1]["saved"] is None
