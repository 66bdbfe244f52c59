"""The embedding's autograd function and the optimizers' clipping without a GPU:
what they pass on, with the library's calls replaced by recorders."""
import pytest
import torch

from bit_blockwise_adamw_gb300 import nn as q8nn
from bit_blockwise_adamw_gb300 import optim

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in ("q8_embedding_forward", "q8_embedding_backward", "q8_grad_norm", "q8_clip_grads", "adamw8bit_sr_step", "adamw_bf16_sr_step",
                 "momentum8bit_sr_step", "lion8bit_sr_step"):
        monkeypatch.setattr(q8nn.B, name, lambda *a, _name=name, **kw: made.append((_name, a, kw)))
    return made


@pytest.mark.parametrize("shape", [(), (5,), (2, 3), (0,), (3, 0)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_embedding_shapes(calls, shape, dtype):
    m = q8nn.Embedding(7, 4, scale=2.0, dtype=dtype)
    ids = torch.zeros(shape, dtype=torch.int64)
    out = m(ids)
    assert out.shape == (*shape, 4) and out.dtype == dtype
    out.sum().backward()
    assert m.weight.grad.shape == (7, 4) and m.weight.grad.dtype == BF
    assert [c[0] for c in calls] == ["q8_embedding_forward", "q8_embedding_backward"]
    assert calls[0][1][0].shape == calls[1][1][0].shape == (ids.numel(),) and calls[1][1][1].shape == (ids.numel(), 4)
    assert calls[0][1][3] == calls[1][1][3] == 2.0


def test_embedding_takes_ids_of_any_layout_and_broadcast_gradients(calls):
    m = q8nn.Embedding(7, 4)
    ids = torch.arange(6).view(2, 3).t()
    out = m(ids)
    assert calls[-1][1][0].tolist() == ids.reshape(-1).tolist() and calls[-1][1][0].is_contiguous()
    out.sum().backward()                             # the gradient of a sum has no strides of its own
    d = calls[-1][1][1]
    assert d.stride() == (4, 1) and d.shape == (6, 4)
    m(ids)[:, :2].sum().backward()


def params(*sizes):
    ps = [torch.nn.Parameter(torch.zeros(n, dtype=BF)) for n in sizes]
    for p in ps:
        p.grad = torch.ones_like(p)
    return ps


def test_clip_grad_norm_passes_the_gradients_that_are_there(calls):
    ps = params(5, 6, 7)
    ps[1].grad = None
    norm = optim.clip_grad_norm_(iter(ps), 2.5)
    (name, a, kw), = calls
    assert name == "q8_clip_grads" and a[1] == 2.5 and a[2] is norm and norm.dim() == 0 and norm.dtype == torch.float32
    assert len(a[0]) == 2 and a[0][0] is ps[0].grad and a[0][1] is ps[2].grad
    optim.clip_grad_norm_(ps[0], float("inf"))
    assert calls[-1][0] == "q8_grad_norm" and len(calls[-1][1][0]) == 1
    ps[0].grad = None
    assert float(optim.clip_grad_norm_(ps[0], 1.0)) == 0 and len(calls) == 2


@pytest.mark.parametrize("cls", [optim.AdamW8bitSR, optim.Momentum8bitSR, optim.Lion8bitSR, optim.AdamWBF16SR])
def test_optimizers_clip_all_groups_together_before_the_step(calls, monkeypatch, cls):
    monkeypatch.setattr(optim, "_check_param", lambda p: p.grad)
    a, b = params(5, 6), params(5000)
    opt = cls([{"params": a}, {"params": b, "lr": 1e-4}], max_grad_norm=0.5)
    assert opt.grad_norm is None
    opt.step()
    assert [c[0] for c in calls][0] == "q8_clip_grads" and len(calls) == 3
    assert [g.numel() for g in calls[0][1][0]] == [5, 6, 5000] and calls[0][1][1] == 0.5 and calls[0][1][2] is opt.grad_norm
    calls.clear()
    plain = cls([{"params": a}, {"params": b}])
    plain.step()
    assert len(calls) == 2 and not any("clip" in c[0] for c in calls) and plain.grad_norm is None
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="max_grad_norm"):
            cls(a, max_grad_norm=bad)


def test_closures_run_before_clipping(calls, monkeypatch):
    monkeypatch.setattr(optim, "_check_param", lambda p: p.grad)
    ps = params(5)
    opt = optim.AdamW8bitSR(ps, max_grad_norm=1.0)

    def closure():
        ps[0].grad = torch.full_like(ps[0], 3.0)
        return torch.tensor(7.0)
    assert float(opt.step(closure)) == 7.0
    assert calls[0][1][0][0] is ps[0].grad
