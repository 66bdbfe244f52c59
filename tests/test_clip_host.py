"""Clipping through clip_grad_norm_ and the optimizers without a GPU, the
library's calls replaced by recorders: what may be refused is refused before a
gradient is touched, and no gradient is passed twice."""
import pytest
import torch

from bit_blockwise_adamw_gb300 import optim

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in ("q8_grad_norm", "q8_clip_grads", "adamw8bit_sr_step", "adamw_bf16_sr_step", "momentum8bit_sr_step", "lion8bit_sr_step"):
        monkeypatch.setattr(optim.B, name, lambda *a, _name=name, **kw: made.append((_name, a, kw)))
    return made


def params(*sizes):
    ps = [torch.nn.Parameter(torch.zeros(n, dtype=BF)) for n in sizes]
    for p in ps:
        p.grad = torch.ones_like(p)
    return ps


@pytest.mark.parametrize("limit", [1.0, float("inf")])
def test_a_repeated_parameter_counts_and_is_clipped_once(calls, limit):
    """As from two modules with a tied weight: its gradient in two places of the
    list would be scaled by two CTAs, in no order."""
    a, b = params(5, 6)
    optim.clip_grad_norm_([a, b, a, a], limit)
    passed = calls[0][1][0]
    assert len(passed) == 2 and passed[0] is a.grad and passed[1] is b.grad
