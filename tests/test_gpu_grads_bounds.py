"""How exact the norm of all gradients is, at the numbers of elements and of
tensors where a sum in plain float32 would not be.

Tolerances.  u = 2^-24, half a step of float32.  Of the sum of squares, a thread
adds its elements in four chains, of 16 squares each for bf16 and of 8 for
float32, each addition rounding by u, and the four in two more: (16 + 2) u or
(8 + 2) u.  Pairs of floats and whole numbers keep what follows (2^-26 of the sum
is more than they lose below 2^34 elements); the sum is rounded once, by u.  Half
of that reaches the norm, whose root is rounded once: 1.5 u beside the chains'.
The factor adds the rounding of max_norm, of norm + 1e-6 and of the quotient, the
result its own."""
import math

import numpy as np
import pytest
import torch

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
EXACT = (1.5 + 2.0 ** -3) * U                       # where the chains are exact
CHAINS = {BF: EXACT + 9 * U, F32: EXACT + 5 * U}

PARTS = 456                                         # CTAs of one launch on 152 SMs, and tensors of a launch
PER_LAUNCH = 768
LONG = 150 * PER_LAUNCH                             # 150 launches of short tensors
VALUE = 239 / 128                                   # its square has 16 bits: sums of 100 are exact in float32

FLAT = 321 * PARTS * 8192                           # a thread adds 321 sums of 32 squares
FLAT_VALUE = 981 / 1024                             # its square has 20 bits: sums of 32 are exact, those of 321 times as many are not


def f32(x):
    return np.asarray(x, np.float32)


def test_plain_sums_would_leave_these_bounds():
    """What the GPU tests below stand for: the same sums in plain float32, one
    after the other, miss their tolerances by far."""
    total = np.float32(0)
    for _ in range(321):
        total = np.float32(total + np.float32(32 * FLAT_VALUE ** 2))
    want = 321 * 32 * FLAT_VALUE ** 2
    assert abs(math.sqrt(float(total)) / math.sqrt(want) - 1) > 10 * EXACT
    s = 100 * VALUE ** 2                            # a launch's sums: two tensors to a CTA, then one
    parts = np.tile(np.array([2 * s] * (PER_LAUNCH - PARTS) + [s] * (2 * PARTS - PER_LAUNCH)), LONG // PER_LAUNCH)
    threads = np.zeros(256, np.float32)
    for at in range(0, len(parts), 256):
        some = f32(parts[at:at + 256])
        threads[:len(some)] = f32(threads[:len(some)] + some)
    got = math.sqrt(float(threads.astype(np.float64).sum()))
    assert abs(got / math.sqrt(parts.sum()) - 1) > 5 * EXACT


def new_norm():
    return torch.full((1,), -1.0, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lists_of_many_launches(cuda_device, dtype):
    """The norm of more than a hundred thousand tensors, and their clipping."""
    import bit_blockwise_adamw_gb300 as q8
    g = torch.full((100,), VALUE, dtype=dtype, device="cuda")
    want, norm = math.sqrt(LONG * 100) * VALUE, new_norm()
    q8.q8_grad_norm([g] * LONG, norm)
    assert abs(float(norm) - want) <= EXACT * want, (float(norm) / want - 1) / U
    flat = torch.full((LONG * 100,), VALUE, dtype=dtype, device="cuda")
    out = torch.empty(LONG * 100, dtype=F32, device="cuda")
    again = new_norm()
    q8.q8_clip_grads(flat.split(100), 10.0, again, out=out.split(100))
    assert torch.equal(again, norm)
    c = 10.0 / (want + 1e-6)
    assert bool(((out.double() - VALUE * c).abs() <= VALUE * c * (EXACT + 4 * U)).all())
    q8.q8_clip_grads(flat.split(100), 10.0, again)
    assert torch.equal(flat, out.to(dtype))


@pytest.mark.gpu
def test_a_thread_that_adds_many_equal_sums(cuda_device):
    import bit_blockwise_adamw_gb300 as q8
    g, norm = torch.full((FLAT,), FLAT_VALUE, device="cuda"), new_norm()
    q8.q8_grad_norm([g], norm)
    want = math.sqrt(FLAT) * FLAT_VALUE
    assert abs(float(norm) - want) <= EXACT * want, (float(norm) / want - 1) / U


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [[1], [100, 7], [1 << 20], [16385, 65537, 3], [9000001, 3, 7000003, 16385], [60000001]])
def test_norm_to_its_chains_roundings(cuda_device, dtype, sizes):
    import bit_blockwise_adamw_gb300 as q8
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    for std in (1e-30, 1e-3, 1.0, 1e15):
        grads = [(torch.randn(n, generator=gen, device="cuda") * std * (1 + i)).to(dtype) for i, n in enumerate(sizes)]
        norm = new_norm()
        q8.q8_grad_norm(grads, norm)
        want = math.sqrt(sum(float((g.double() / std).square().sum()) for g in grads)) * std
        tol = CHAINS[dtype] if std not in (1e-30, 1e15) else EXACT + 32 * U      # squares out of range: one chain of up to 64
        assert abs(float(norm) - want) <= tol * want, (std, (float(norm) / want - 1) / U)
