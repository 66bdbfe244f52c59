"""The norm of all gradients and their clipping on the GPU, against float64.

Tolerances.  Squares are added in float32 over at most 128 elements, each
addition rounding by 2^-24 of sums of positive terms: 128 * 2^-24 of the sum of
squares, half of it of the norm, and 2^-24 for the norm's own rounding; 66 * 2^-24
in all.  The factor carries the norm's error before its rounding and a rounding
of its own, the result one more and half a step of its type."""
import math
import os
import subprocess
import sys

import pytest
import torch

import bit_blockwise_adamw_gb300 as q8

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32
NORM_TOL = 66 * 2.0 ** -24
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -133, F32: 2.0 ** -149}


def rnd(n, seed=0, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def norm_of(grads):
    """In float64, from values scaled by their largest: no square leaves its range."""
    top = max([float(g.double().abs().max()) for g in grads if g.numel()] or [0.0])
    if top == 0 or not math.isfinite(top):
        return top
    return math.sqrt(sum(float((g.double() / top).square().sum()) for g in grads)) * top


def new_norm():
    return torch.full((1,), -1.0, device="cuda")


def check_clipped(grads, outs, limit, norm):
    c = min(1.0, limit / (norm + 1e-6))
    for g, o in zip(grads, outs):
        want = g.double() * c
        off = (o.double() - want).abs()
        assert bool((off <= want.abs() * (U[o.dtype] + 69 * 2.0 ** -24) + TINY[o.dtype]).all()), float(off.max())


LISTS = {
    "one element": [1],
    "one": [1 << 20],
    "short": [1, 2, 3, 5, 7, 8, 9, 31, 33, 63, 65, 127, 129, 1000, 1023, 1025],
    "with empty ones": [0, 5, 0, 0, 70000, 0],
    "chunk edges": [16383, 16384, 16385, 32767, 32768, 32769, 65535, 65537, 131071, 131073],
    "many": [(i * 37) % 5000 + 1 for i in range(1700)],
    "a long one among short ones": [64, 3000001, 64, 1, 2000000],
    "more chunks than parts": [9000001, 3, 7000003, 16385, 12000001, 5],
    "several chunks to a CTA": [20000001, 77, 30000005, 4097],
}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("which", LISTS)
def test_norm_and_clipping(cuda_device, which, dtype):
    grads = [rnd(n, seed=i, std=1e-2 * (1 + i % 7), dtype=dtype) for i, n in enumerate(LISTS[which])]
    want = norm_of(grads)
    norm = new_norm()
    q8.q8_grad_norm(grads, norm)
    assert abs(float(norm) - want) <= NORM_TOL * want
    for limit in (0.25 * want, 4 * want, 0.0, math.inf):
        for out_dtype in (BF, F32):
            outs = [torch.full_like(g, float("nan"), dtype=out_dtype) for g in grads]
            clipped = new_norm()
            q8.q8_clip_grads(grads, limit, clipped, out=outs)
            assert torch.equal(clipped, norm), "the same bits as the norm alone"
            check_clipped(grads, outs, limit, want)
        mine = [g.clone() for g in grads]
        q8.q8_clip_grads(mine, limit, clipped)
        for m, o in zip(mine, outs if dtype == F32 else [o.to(BF) for o in outs]):
            assert torch.equal(m, o), "in place, as elsewhere"
        if limit > want:
            assert all(torch.equal(m, g) for m, g in zip(mine, grads))


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_alignment_and_what_lies_between(cuda_device, dtype, out_dtype):
    """Tensors at every element's alignment, inputs and outputs apart; what lies
    around them is neither counted nor written."""
    for shift in range(9):
        src = torch.full((80000,), float("nan"), dtype=dtype, device="cuda")
        dst = torch.full((80000,), 7.0, dtype=out_dtype, device="cuda")
        grads, outs, written = [], [], torch.zeros(80000, dtype=torch.bool, device="cuda")
        at = 16
        for i, n in enumerate((1, 7, 100, 1000, 16384, 40001)):
            a, b = at + shift, at + (shift * 3 + i) % 11
            src[a:a + n] = rnd(n, seed=i, dtype=dtype)
            grads.append(src[a:a + n])
            outs.append(dst[b:b + n])
            written[b:b + n] = True
            at += n + 30
        want, norm = norm_of(grads), new_norm()
        q8.q8_clip_grads(grads, 1.0, norm, out=outs)
        assert abs(float(norm) - want) <= NORM_TOL * want
        check_clipped(grads, outs, 1.0, want)
        assert bool((dst[~written] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [[5], [300], [40000, 20000], [200000]])
def test_magnitudes(cuda_device, dtype, sizes):
    """From the smallest subnormal numbers to the largest ones, alone and mixed,
    with zeros among them."""
    top, low = (3.0e38, 2.0 ** -133) if dtype == BF else (3.4e38, 2.0 ** -149)
    for std in (0.0, low, 1e-38, 1e-30, 1e-24, 1e-19, 1e-12, 1.0, 1e12, 1e18, 1e25, 1e35):
        grads = [rnd(n, seed=i, std=std, dtype=dtype) if std != low else torch.full((n,), low, dtype=dtype, device="cuda")
                 for i, n in enumerate(sizes)]
        for g in grads:
            g[::3] = 0
            if g.numel() > 100:
                g[64:] *= 2.0 ** -60 if std >= 1e-12 else 1.0       # far below the others: lost beside them, rightly
        want, norm = norm_of(grads), new_norm()
        q8.q8_grad_norm(grads, norm)
        assert abs(float(norm) - want) <= NORM_TOL * want + TINY[F32], (std, float(norm), want)
    grads = [torch.full((n,), top, dtype=dtype, device="cuda") for n in sizes]
    want, norm = norm_of(grads), new_norm()
    q8.q8_grad_norm(grads, norm)
    assert float(norm) == math.inf if want > 3.41e38 else abs(float(norm) - want) <= NORM_TOL * want
    tiny = [torch.zeros(n, dtype=dtype, device="cuda") for n in sizes]
    tiny[-1][-1] = low
    q8.q8_grad_norm(tiny, norm)
    assert float(norm) == low


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_that_are_not_finite(cuda_device, dtype):
    for n in (3, 70000):
        for bad in (math.inf, -math.inf, math.nan):
            grads = [rnd(n, seed=1, dtype=dtype), rnd(100, seed=2, dtype=dtype)]
            grads[0][n // 2] = bad
            norm, outs = new_norm(), [torch.empty_like(g) for g in grads]
            q8.q8_clip_grads(grads, 1.0, norm, out=outs)
            nan = math.isnan(bad)
            assert math.isnan(float(norm)) if nan else float(norm) == math.inf
            if nan:
                assert all(bool(o.isnan().all()) for o in outs)
            else:
                assert bool(outs[0][n // 2].isnan()) and int(outs[0].isnan().sum()) == 1 and not outs[1].any()
                assert bool((outs[0][:n // 2] == 0).all())


def test_nothing_to_do(cuda_device):
    norm = new_norm()
    q8.q8_grad_norm([], norm)
    assert float(norm) == 0
    norm = new_norm()
    q8.q8_clip_grads([torch.empty(0, dtype=BF, device="cuda")], 1.0, norm)
    assert float(norm) == 0
    zeros = [torch.zeros(1000, dtype=BF, device="cuda")]
    q8.q8_clip_grads(zeros, 1.0, norm)
    assert float(norm) == 0 and not zeros[0].any()


def test_types_mixed_in_one_list_and_packed(cuda_device):
    grads = [rnd(70001, seed=1, dtype=F32), rnd(3001, seed=2), rnd(5, seed=3, dtype=F32).view(5, 1), rnd(12 * 7, seed=4).view(12, 7)]
    outs = [torch.empty_like(g, dtype=BF) for g in grads]
    want, norm = norm_of(grads), new_norm()
    packed = q8.pack_grads(grads, outs)
    for _ in range(2):
        q8.q8_clip_grads(packed, 1.0, norm)
        assert abs(float(norm) - want) <= NORM_TOL * want
        check_clipped(grads, outs, 1.0, want)
        grads[0].mul_(0.5)                            # the packed list says where the gradients are, not what they hold
        want = norm_of(grads)
    q8.q8_grad_norm(packed, norm)
    assert abs(float(norm) - want) <= NORM_TOL * want
    with pytest.raises(ValueError, match="packed"):
        q8.q8_clip_grads(packed, 1.0, norm, out=outs)
    with pytest.raises(ValueError, match="number of elements"):
        q8.pack_grads(grads, outs[:2])
    with pytest.raises(ValueError, match="one float32"):
        q8.q8_grad_norm(grads, torch.zeros(2, device="cuda"))
    with pytest.raises(q8.Q8Error, match="type"):
        q8.q8_clip_grads([grads[0]], 1.0, norm, out=[grads[0].view(BF)[:70001]])


def test_offsets_past_32_bits(cuda_device):
    """One gradient of more than 2^31 elements; only its ends are not zero."""
    n = (1 << 31) + 70003
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[0], g[-1], g[1 << 31] = 3.0, 4.0, 12.0
    norm = new_norm()
    q8.q8_clip_grads([g], 1.0, norm)
    assert float(norm) == 13.0
    c = 1.0 / (13.0 + 1e-6)
    for i, x in ((0, 3.0), (-1, 4.0), (1 << 31, 12.0)):
        assert abs(float(g[i]) - x * c) <= x * c * 2.0 ** -8
    assert int(torch.count_nonzero(g)) == 3


def test_other_streams_and_workspaces(cuda_device):
    a, b = [rnd(3000000, seed=1), rnd(7, seed=2)], [rnd(2000001, seed=3, std=5.0)]
    want = [new_norm(), new_norm()]
    for g, w in zip((a, b), want):
        q8.q8_grad_norm(g, w)
    ws = torch.empty(q8.q8_grad_norm_workspace(1), dtype=torch.uint8, device="cuda").random_(0, 255)
    got, outs = [new_norm(), new_norm()], [torch.empty_like(b[0])]
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(one):
            q8.q8_grad_norm(a, got[0])
        q8.q8_clip_grads(b, 1.0, got[1], out=outs, workspace=ws, stream=two)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_clipped(b, outs, 1.0, norm_of(b))


CHILD = r"""
import torch
import bit_blockwise_adamw_gb300 as q8
q8.q8_prepare_device()
g = torch.Generator(device="cuda").manual_seed(1)
for sizes in ([1000], [64] * 900, [5000000, 3, 70001]):
    grads = [torch.randn(n, generator=g, device="cuda").bfloat16() for n in sizes]
    a, b = ([torch.empty_like(x) for x in grads] for _ in "ab")
    na, nb, only = (torch.empty(1, device="cuda") for _ in "abc")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.q8_clip_grads(grads, 1.0, na, out=a)
        q8.q8_grad_norm(grads, only)
    for scale in (1.0, 0.0, 1e-30, 3.0):             # replayed, and replayed on other values
        for x in grads:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * scale)
        graph.replay()
        q8.q8_clip_grads(grads, 1.0, nb, out=b)
        torch.cuda.synchronize()
        assert torch.equal(na, nb) and torch.equal(only, nb)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
print("OK")
"""


def test_captured_in_a_graph_after_prepare(cuda_device):
    env = dict(os.environ)
    env["PYTHONPATH"] = os.pathsep.join([ROOT, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
