"""The autograd functions and modules over the training-step operators: the
gradients that reach the parameters are the operators' own, a small step runs
end to end with the optimizer, and the calls are captured in a CUDA graph."""
import os
import subprocess
import sys

import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import nn as q8nn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def rnd(*shape, seed=0, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("recompute", [False, True])
def test_gated_ff_is_the_operator(cuda_device, recompute):
    x, wg, wu = (rnd(*s, seed=i, std=0.1).requires_grad_() for i, s in enumerate(((2, 35, 72), (136, 72), (136, 72))))
    h = q8nn.gated_ff(x, wg, wu, "gelu", recompute)
    dh = rnd(2, 35, 136, seed=9)
    dx, dwg, dwu = torch.autograd.grad(h, (x, wg, wu), dh)
    flat = x.detach().view(70, 72)
    want = [torch.empty_like(t) for t in (flat, dwg, dwu)]
    saved = None if recompute else torch.empty(2, 70, 136, device="cuda")
    if saved is not None:
        q8.q8_gated_ff_forward(flat, wg.detach(), wu.detach(), torch.empty(70, 136, dtype=BF, device="cuda"), q8.GELU, saved=saved)
    q8.q8_gated_ff_backward(flat, wg.detach(), wu.detach(), dh.view(70, 136), *want, q8.GELU, saved=saved)
    for got, w in zip((dx.view(70, 72), dwg, dwu), want):
        assert torch.equal(got, w)
    only, = torch.autograd.grad(q8nn.gated_ff(x, wg, wu, "gelu", recompute), wu, dh)
    assert torch.equal(only, dwu)


def test_block_norm_grads_and_unused_outputs(cuda_device):
    m = q8nn.BlockNorm(96, post="layer", pre="rms", residual_scale=0.5, device="cuda")
    r, y = rnd(3, 11, 96, seed=1, dtype=torch.float32).requires_grad_(), rnd(3, 11, 96, seed=2).requires_grad_()
    out, z = m(r, y)
    assert out.dtype == torch.float32 and z.dtype == BF and out.shape == r.shape
    both = torch.autograd.grad((out.sum() + z.float().square().sum()), [r, y, *m.parameters()], retain_graph=True)
    only_z = torch.autograd.grad(z.float().square().sum(), [r, y, *m.parameters()], retain_graph=True)
    only_r = torch.autograd.grad(out.sum(), [r, y], retain_graph=True)
    assert torch.allclose(both[0], only_z[0] + only_r[0], rtol=1e-4, atol=1e-4)
    assert all(g.shape == p.shape for g, p in zip(both[2:], m.parameters()))


def test_distill_gradient_scales_with_the_upstream(cuda_device):
    z = rnd(2, 9, 777, seed=3, dtype=torch.float32).requires_grad_()
    teacher = rnd(2, 9, 777, seed=4, std=3.0, dtype=torch.float32)
    t, ids = teacher.topk(12, -1)
    loss = q8nn.distill_topk(z, ids, t, labels=ids[..., 0], temperature=2.0, kd_weight=0.5, ce_weight=0.5)
    assert loss.shape == (2, 9) and loss.dtype == torch.float32
    w = torch.rand(2, 9, device="cuda")
    g, = torch.autograd.grad((loss * w).sum(), z, retain_graph=True)
    fused = torch.empty(18, 777, device="cuda")
    q8.q8_distill_topk_forward(z.detach().view(18, 777), ids.view(18, 12), t.view(18, 12), torch.empty(18, device="cuda"),
                               labels=ids[..., 0].reshape(18).contiguous(), row_weight=w.view(18), dlogits=fused,
                               temperature=2.0, kd_weight=0.5, ce_weight=0.5)
    assert torch.allclose(g.view(18, 777), fused, rtol=2e-5, atol=1e-7)


def test_example_learns(cuda_device):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import distill_step
    finally:
        sys.path.pop(0)
    losses = distill_step.train(steps=80)
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    assert last < 0.7 * first, (first, last)


CHILD = r"""
import torch
import bit_blockwise_adamw_gb300 as q8
q8.q8_prepare_device()
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()
E = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")

def step(T, o):
    x, wg, wu, dh, y, w, z, ids, t, lab = o["in"]
    q8.q8_gated_ff_forward(x, wg, wu, o["h"], saved=o["saved"], workspace=o["ws"])
    q8.q8_gated_ff_backward(x, wg, wu, dh, o["dx"], o["dwg"], o["dwu"], saved=o["saved"], workspace=o["ws"])
    q8.q8_block_norm_forward(x, y, o["ro"], o["z"], 1, 2, post_weight=w, gate=w)
    q8.q8_block_norm_backward(x, y, o["ro"], o["z"], o["dr"], o["dy"], 1, 2, post_weight=w, gate=w, dgate=o["dgate"],
                              dpost_weight=o["dpw"], workspace=o["ws"])
    q8.q8_distill_topk_forward(z, ids, t, o["loss"], dlogits=o["dz"], labels=lab, temperature=2.0, kd_weight=.5, ce_weight=.5)

def outputs(T, D, F, V, K, ins):
    return {"in": ins, "h": E(T, F), "saved": E(2, T, F, dtype=torch.float32), "ws": E(1 << 26, dtype=torch.uint8), "dx": E(T, D),
            "dwg": E(F, D), "dwu": E(F, D), "ro": E(T, D), "z": E(T, D), "dr": E(T, D), "dy": E(T, D), "dgate": E(D), "dpw": E(D),
            "loss": E(T, dtype=torch.float32), "dz": E(T, V)}

for T, D, F, V, K in ((70, 136, 264, 3001, 9), (300, 512, 1032, 50257, 33)):
    ins = (r(T, D), r(F, D, std=.05), r(F, D, std=.05), r(T, F), r(T, D), r(D), r(T, V, std=3.0),
           torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(T)]),
           torch.randn(T, K, generator=g, device="cuda"), torch.randint(0, V, (T,), generator=g, device="cuda"))
    a, b = outputs(T, D, F, V, K, ins), outputs(T, D, F, V, K, ins)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(T, a)
    graph.replay()
    step(T, b)
    torch.cuda.synchronize()
    for k in a:
        if k not in ("in", "ws"):
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
print("OK")
"""


def test_captured_in_a_graph_after_prepare(cuda_device):
    env = dict(os.environ)
    env["PYTHONPATH"] = os.pathsep.join([ROOT, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
