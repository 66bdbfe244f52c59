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
