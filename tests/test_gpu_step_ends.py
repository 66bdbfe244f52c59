"""The embedding, the clipping and what lies between them, as a training step
uses them: autograd, the optimizers' max_grad_norm, a captured step."""
import os
import subprocess
import sys

import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import nn as q8nn
from bit_blockwise_adamw_gb300 import optim

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def rnd(*shape, seed=0, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_embedding_is_the_operator(cuda_device, dtype):
    m = q8nn.Embedding(501, 72, scale=3.0, dtype=dtype, device="cuda")
    ids = torch.randint(-3, 510, (4, 33), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    out = m(ids)
    want = torch.empty(132, 72, dtype=dtype, device="cuda")
    q8.q8_embedding_forward(ids.view(-1), m.weight.detach(), want, scale=3.0)
    assert torch.equal(out.detach().view(132, 72), want)
    d = rnd(4, 33, 144, seed=2, dtype=dtype)[..., :72]           # rows that are not contiguous
    out.backward(d)
    dw = torch.empty(501, 72, dtype=BF, device="cuda")
    q8.q8_embedding_backward(ids.view(-1), d.reshape(132, 72), dw, scale=3.0)
    assert torch.equal(m.weight.grad, dw)
    m(ids).backward(d)                                           # autograd adds a second one
    assert torch.equal(m.weight.grad, dw + dw)
    with torch.inference_mode():
        assert torch.equal(m(ids), out)


def test_tied_weights_by_accumulation(cuda_device):
    """The output layer's gradient first, the embedding's added to it: the same
    as their sum, rounded once."""
    ids = torch.randint(0, 50, (300,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    head, d = rnd(999, 64, seed=1), rnd(300, 64, seed=2)
    got = head.clone()
    q8.q8_embedding_backward(ids, d, got, accumulate=True)
    want = head.double().index_add_(0, ids, d.double())
    size = head.double().abs().index_add_(0, ids, d.double().abs())
    n = torch.bincount(ids, minlength=999).double()[:, None]
    assert bool(((got.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * (n + 1) * 2.0 ** -24).all())


def params(sizes, seed=0):
    return [torch.nn.Parameter(rnd(*s, seed=seed + i, std=0.02)) for i, s in enumerate(sizes)]


@pytest.mark.parametrize("cls", [optim.AdamW8bitSR, optim.Momentum8bitSR, optim.Lion8bitSR, optim.AdamWBF16SR])
@pytest.mark.parametrize("limit", [0.05, 1e9])
def test_max_grad_norm_is_clipping_and_a_step(cuda_device, cls, limit):
    sizes = [(300, 64), (64,), (4096,), (1000, 7)]
    a, b = params(sizes), params(sizes)
    one = cls([{"params": a[:2]}, {"params": a[2:]}], seed=3, max_grad_norm=limit)
    two = cls([{"params": b[:2]}, {"params": b[2:]}], seed=3)
    for step in range(3):
        for i, (p, q) in enumerate(zip(a, b)):
            p.grad = rnd(*p.shape, seed=100 * step + i, std=1e-3 * (i + 1))
            q.grad = p.grad.clone()
        want = torch.stack([p.grad.double().square().sum() for p in a]).sum().sqrt()
        one.step()
        assert abs(float(one.grad_norm) - float(want)) <= float(want) * 66 * 2.0 ** -24
        norm = torch.empty(1, device="cuda")
        q8.q8_clip_grads([q.grad for q in b], limit, norm)
        two.step()
        for p, q in zip(a, b):
            assert torch.equal(p.grad, q.grad) and torch.equal(p.detach(), q.detach())


def test_clip_grad_norm_(cuda_device):
    sizes = [(64, 33), (1000,), (5,)]
    a, b = params(sizes), params(sizes)
    for i, (p, q) in enumerate(zip(a, b)):
        p.grad = rnd(*p.shape, seed=i, std=0.3)
        q.grad = p.grad.clone()
    got = optim.clip_grad_norm_(a, 0.7)
    want = torch.stack([q.grad.double().square().sum() for q in b]).sum().sqrt()
    assert abs(float(got) - float(want)) <= float(want) * 66 * 2.0 ** -24
    c = 0.7 / (float(want) + 1e-6)
    for p, q in zip(a, b):
        assert bool(((p.grad.double() - q.grad.double() * c).abs() <= q.grad.double().abs() * c * (2.0 ** -8 + 69 * 2.0 ** -24)).all())


CHILD = r"""
import torch
import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import nn as q8nn

q8.q8_prepare_device()
BF = torch.bfloat16
V, D, F, T = 3001, 136, 264, 700
g = torch.Generator(device="cuda").manual_seed(1)
R = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(BF)
ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
dh = R(T, F, std=1e-2)
weights = [R(V, D, std=0.02), R(F, D, std=0.05), R(F, D, std=0.05)]

# one step: lookup, feed-forward, their gradients, clipping, the 8-bit update
def step(w, s, hp):
    q8.q8_embedding_forward(ids, w[0], s["x"], scale=8.0)
    q8.q8_gated_ff_forward(s["x"], w[1], w[2], s["h"], saved=s["saved"])
    q8.q8_gated_ff_backward(s["x"], w[1], w[2], dh, s["dx"], s["g"][1], s["g"][2], saved=s["saved"])
    q8.q8_embedding_backward(ids, s["dx"], s["g"][0], scale=8.0)
    q8.q8_clip_grads(s["g"], 0.1, s["norm"])
    q8.adamw8bit_sr_step(s["t"], hp)

def state():
    w = [x.clone() for x in weights]
    E = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")
    grads = [torch.empty_like(x) for x in w]
    tensors = [q8.Tensor8.zeros_like(x.view(-1), y.view(-1)) for x, y in zip(w, grads)]
    return w, {"x": E(T, D), "h": E(T, F), "saved": E(2, T, F, dtype=torch.float32), "dx": E(T, D), "g": grads,
               "norm": E(1, dtype=torch.float32), "t": tensors}

hp = q8.hparams(lr=1e-3, weight_decay=0.1, step=1, seed=5)
a, b = state(), state()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step(*a, hp)
for _ in range(3):
    graph.replay()
    step(*b, hp)
torch.cuda.synchronize()
assert float(a[1]["norm"]) > 0.1
for x, y in zip(a[0] + a[1]["g"] + [a[1]["norm"]], b[0] + b[1]["g"] + [b[1]["norm"]]):
    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
assert not any(torch.equal(x, y) for x, y in zip(a[0], weights))
clipped = torch.stack([x.double().square().sum() for x in a[1]["g"]]).sum().sqrt()
# each element is off by at most half a step of bf16, and so is their norm; the factor by 70 * 2^-24 and the 1e-6
assert abs(float(clipped) - 0.1) < 0.1 * (2.0 ** -8 + 1e-4), float(clipped)
print("OK")
"""


def test_a_whole_step_captured_in_a_graph(cuda_device):
    env = dict(os.environ)
    env["PYTHONPATH"] = os.pathsep.join([ROOT, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


def test_example_trains_its_embedding(cuda_device):
    """The example runs, and its embedding's gradient is the formula's."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import distill_step
    finally:
        sys.path.pop(0)
    assert len(distill_step.train(steps=3)) == 3
    torch.manual_seed(0)
    student = distill_step.Student(203, 64, 128, 1, 2, "cuda")
    tokens = torch.randint(0, 203, (50, 2), device="cuda")
    rows = {}
    student.embed.register_forward_hook(lambda m, i, o: o.register_hook(lambda d: rows.update(d=d)) and None)
    student(tokens).float().square().sum().backward()
    got, d = student.embed.weight.grad.double(), rows["d"].double().view(100, 64)
    want = torch.zeros(203, 64, dtype=torch.float64, device="cuda").index_add_(0, tokens.view(-1), d)
    size = torch.zeros(203, 64, dtype=torch.float64, device="cuda").index_add_(0, tokens.view(-1), d.abs())
    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -8 + size * 100 * 2.0 ** -24 + 2.0 ** -133).all())
