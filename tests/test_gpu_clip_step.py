"""Clipping steps on the GPU: captured and replayed, refused, and with a parameter
that comes twice."""
import math

import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import optim

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
OPTIMIZERS = [optim.AdamW8bitSR, optim.Momentum8bitSR, optim.Lion8bitSR, optim.AdamWBF16SR]


def rnd(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def params(seed=0):
    return [torch.nn.Parameter(rnd(*s, seed=seed + i, std=0.02)) for i, s in enumerate([(300, 64), (64,), (4096,), (1000, 7)])]


def set_grads(ps, seed, std=0.1):
    for i, p in enumerate(ps):
        g = rnd(*p.shape, seed=seed + i, std=std)
        if p.grad is None:
            p.grad = g
        else:
            p.grad.copy_(g)


@pytest.mark.parametrize("cls", OPTIMIZERS)
def test_a_captured_step_clips_as_an_eager_one(cuda_device, cls):
    """A captured step keeps the step counter that it was captured with; the twin
    is given the same one."""
    a, b = params(), params()
    one, two = (cls([{"params": p[:2]}, {"params": p[2:]}], seed=3, max_grad_norm=0.5) for p in (a, b))
    for ps, opt in ((a, one), (b, two)):
        set_grads(ps, 10)
        opt.step()                                   # its state is made by the first step
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.step()
    for replay in range(3):
        set_grads(a, 100 * (replay + 1))
        set_grads(b, 100 * (replay + 1))
        graph.replay()
        for group in two.param_groups:
            group["step"] = 1
        two.step()
        torch.cuda.synchronize()
        assert torch.equal(one.grad_norm, two.grad_norm) and float(one.grad_norm) > 0.5
        for p, q in zip(a, b):
            assert torch.equal(p.grad, q.grad) and torch.equal(p.detach(), q.detach())


@pytest.mark.parametrize("cls", OPTIMIZERS)
def test_a_refused_step_leaves_gradients_and_parameters(cuda_device, cls):
    ps = params()
    opt = cls([{"params": ps[:2]}, {"params": ps[2:]}], max_grad_norm=1e-3)
    set_grads(ps, 5)
    buf = torch.zeros(7009, dtype=BF, device="cuda")
    ps[3].grad = buf[1:7001].view(1000, 7).copy_(ps[3].grad)          # off 16 bytes
    before = [(p.grad.clone(), p.detach().clone()) for p in ps]
    with pytest.raises(ValueError, match="aligned"):
        opt.step()
    for p, (g, w) in zip(ps, before):
        assert torch.equal(p.grad, g) and torch.equal(p.detach(), w)
    assert opt.grad_norm is None


def test_a_repeated_parameter(cuda_device):
    a, b = params()[:2]
    set_grads([a, b], 7)
    want = math.sqrt(float(a.grad.double().square().sum() + b.grad.double().square().sum()))
    before = a.grad.clone()
    norm = optim.clip_grad_norm_([a, b, a, b, a], want / 4)
    assert abs(float(norm) - want) <= 11 * 2.0 ** -24 * want
    c = 1 / 4                                        # the 1e-6 and the roundings of norm and factor: below 2^-20 of it
    assert bool(((a.grad.double() - before.double() * c).abs() <= before.double().abs() * c * (2.0 ** -8 + 2.0 ** -17)).all())


def test_the_same_tensor_twice_is_refused(cuda_device):
    g, norm = rnd(5000), torch.zeros(1, device="cuda")
    for grads, out in (([g, g], None), ([g, g[10:20]], None), ([rnd(8), rnd(8)], [g[:8], g[4:12]]), ([g[:8], rnd(8)], [rnd(8), g[7:15]])):
        with pytest.raises(q8.Q8Error, match="overlap"):
            q8.q8_clip_grads(grads, 1.0, norm, out=out)
    before = g.clone()
    q8.q8_grad_norm([g, g], norm)
    assert torch.equal(g, before) and abs(float(norm) - math.sqrt(2 * float(g.double().square().sum()))) <= 11 * 2.0 ** -24 * float(norm)
