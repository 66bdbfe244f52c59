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


class OnGpu(torch.Tensor):
    """A CPU tensor that says that it is on a GPU."""
    is_cuda = True


def refused_params():
    """Two groups' parameters, the last one's gradient of a type that clipping takes and no step."""
    ps = [torch.nn.Parameter(torch.zeros(n, dtype=BF).as_subclass(OnGpu)) for n in (5, 6, 5000)]
    for p in ps:
        p.grad = torch.ones(p.shape, dtype=BF)
    return ps


OPTIMIZERS = [optim.AdamW8bitSR, optim.Momentum8bitSR, optim.Lion8bitSR, optim.AdamWBF16SR]


@pytest.fixture
def prepared(monkeypatch):
    monkeypatch.setattr(optim.B, "q8_prepare_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "device", lambda d: torch.autograd.profiler.record_function("device"))


@pytest.mark.parametrize("cls", OPTIMIZERS)
@pytest.mark.parametrize("fault,limit", [("type", None), ("type", 0.5), ("layout", None), ("layout", 0.5), ("alignment", 0.5)])
def test_a_refused_step_touches_nothing(calls, prepared, cls, limit, fault):
    ps = refused_params()
    empty = torch.nn.Parameter(torch.zeros(9, dtype=BF)[1:1].as_subclass(OnGpu))      # at no alignment, of no elements
    empty.grad = torch.ones(9, dtype=BF)[1:1]
    opt = cls([{"params": [*ps[:2], empty]}, {"params": ps[2:]}], max_grad_norm=limit)
    opt.step()
    assert len(calls) == (3 if limit else 2)
    calls.clear()
    before = opt.grad_norm
    bad = {"type": lambda: torch.ones(5000), "layout": lambda: torch.ones(10000, dtype=BF)[::2],
           "alignment": lambda: torch.ones(5008, dtype=BF)[1:5001]}[fault]()
    if fault == "type":                              # torch itself refuses such a gradient but through .data
        ps[2].data = torch.zeros(5000)
        ps[2].grad = bad
        ps[2].data = torch.zeros(5000, dtype=BF)
    else:
        ps[2].grad = bad
    with pytest.raises(ValueError):
        opt.step()
    assert calls == [] and opt.grad_norm is before
    assert [g["step"] for g in opt.param_groups] == [1, 1]


def test_the_norm_of_no_gradients_is_on_the_parameters_device(calls):
    p = torch.nn.Parameter(torch.zeros(5, dtype=BF, device="meta"))
    for given in (p, [p], iter([p, p])):
        norm = optim.clip_grad_norm_(given, 1.0)
        assert norm.device.type == "meta" and norm.dim() == 0 and norm.dtype == torch.float32
    assert float(optim.clip_grad_norm_([], 1.0)) == 0 and calls == []


def test_the_norm_of_no_gradients_is_float32(calls):
    torch.set_default_dtype(torch.float64)
    try:
        assert optim.clip_grad_norm_([torch.nn.Parameter(torch.zeros(3))], 1.0).dtype == torch.float32
    finally:
        torch.set_default_dtype(torch.float32)
