"""Edges of the training-step operators on the GPU: sizes and calls at which a
launch takes another shape, against the float64 forms and within the bounds of
test_gpu_train_ops."""
import math

import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import nn as q8nn
import test_gpu_train_ops as ops
import train_refs as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# ------------------------------------------------------------ gated feed-forward

def test_ff_no_tokens_through_autograd(cuda_device):
    m = q8nn.GatedFeedForward(64, 136, device="cuda")
    out = m(torch.zeros(2, 0, 64, dtype=BF, device="cuda", requires_grad=True))
    assert out.shape == (2, 0, 64)
    out.sum().backward()
    assert all(p.grad is not None and not p.grad.any() for p in m.parameters())


@pytest.mark.parametrize("act", [q8.SILU, q8.GELU_TANH, q8.GELU])
@pytest.mark.parametrize("save", [True, False])
def test_ff_projections_far_past_the_activations_bend(cuda_device, act, save):
    """g of either sign up to 2^100 (its square is past fp32's range): act is g or
    0, its derivative 1 or 0, and nothing is NaN."""
    n = 64
    x = torch.zeros(n, 64, dtype=BF, device="cuda")
    exponent = torch.linspace(20, 100, n // 2).round()
    x[:, 0] = torch.cat([2 ** exponent, -2 ** exponent]).to(BF)
    x[:, 1] = 1.0
    wg, wu = (torch.zeros(64, 64, dtype=BF, device="cuda") for _ in range(2))
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    dh = torch.zeros(n, 64, dtype=BF, device="cuda")
    dh[:, 0] = 1.0
    got = ops.ff_run(x, wg, wu, dh, act, save)
    up = (x[:, :1] > 0).to(BF)
    assert torch.equal(got["h"], (x[:, :1] * up).expand(n, 64))
    assert torch.equal(got["dx"][:, :2], torch.cat([up, x[:, :1] * up], 1)) and not got["dx"][:, 2:].any()
    # dw_up's first element is the sum of the squares, past the type's range
    assert torch.isfinite(got["dwg"]).all() and torch.isinf(got["dwu"][0, 0])
    assert torch.isfinite(got["dwu"].flatten()[1:]).all()


@pytest.mark.parametrize("act", [q8.SILU, q8.GELU_TANH, q8.GELU])
@pytest.mark.parametrize("save", [True, False])
def test_ff_activations_tails_relatively(cuda_device, act, save):
    """g from -12.5 to -4, where act is small: every value within its rounding to
    bf16 relatively, and the mean error of each stretch of g within what is left
    when the roundings (RMS each, independent) cancel.  In fp32 the exponential's
    argument comes to at most 90 with four roundings, 90 * 4 * 2^-24 relative in
    the result, and __expf to 2 + 1.17 * 90 units of 2^-23: together below 2^-14.
    g is a sum of two exact products, each within ACC of it."""
    T, F, few, tiny = 512, 256, 2.0 ** -14, 2.0 ** -120
    x = torch.zeros(T, 64, dtype=BF, device="cuda")
    wg, wu = (torch.zeros(F, 64, dtype=BF, device="cuda") for _ in range(2))
    x[:, 0], x[:, 1], x[:, 2] = torch.linspace(-12.4, -4.1, T), 1.0, 1.0
    wg[:, 0], wg[:, 2], wu[:, 1] = 1.0, torch.linspace(-0.05, 0.05, F), 1.0
    dh = torch.zeros(T, F, dtype=BF, device="cuda")
    dh[:, 0] = 1.0
    got = ops.ff_run(x, wg, wu, dh, act, save)
    g = (x.double() @ wg.double().T).requires_grad_()
    want = R.act(g, act) if act != q8.GELU else 0.5 * g * torch.special.erfc(-g * 0.5 ** 0.5)
    if act == q8.GELU_TANH:                          # (1 + tanh t) / 2 without its cancellation
        want = g * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3))
    slope, = torch.autograd.grad(want.sum(), g, create_graph=True)
    bend, = torch.autograd.grad(slope.sum(), g)
    want, slope, g = want.detach(), slope.detach(), g.detach()
    eg = 2 * ops.ACC * g.abs()
    ops.close(got["h"], want, (ops.U + few) * want.abs() + slope.abs() * eg + tiny, "h")
    # one column of dh: dx's first two columns are the one dg and du, rounded once
    ops.close(got["dx"][:, 0], slope[:, 0], (ops.U + 2 * few) * slope[:, 0].abs() + bend[:, 0].abs() * eg[:, 0] + tiny, "dg")
    ops.close(got["dx"][:, 1], want[:, 0], (ops.U + few) * want[:, 0].abs() + slope[:, 0].abs() * eg[:, 0] + tiny, "du")
    normal = want.abs() > 2.0 ** -100
    off = ((got["h"].double() - want) / want)
    for lo in range(-13, -4):
        at = (g >= lo) & (g < lo + 1) & normal
        n = int(at.sum())
        if n >= 1000:
            slack = few + float((slope.abs() * eg / want.abs())[at].mean()) + 6 * ops.RMS / n ** 0.5
            assert abs(float(off[at].mean())) <= slack, (lo, n, slack)


def test_ff_weights_gradients_over_more_than_2_31_elements(cuda_device):
    """dw sums over every token of dg and du of 135000 x 16384: the first and the
    last weights' rows against float64."""
    T, D, F, n = 135000, 64, 16384, 24
    x, wg, wu, dh = ops.ff_case(T, D, F, seed=6)
    got = ops.ff_run(x, wg, wu, dh, q8.SILU, save=False)
    for rows in (slice(0, n), slice(F - n, F)):
        want, tol = ops.ff_bounds(x, wg[rows], wu[rows], dh[:, rows], q8.SILU)
        for k in ("dwg", "dwu"):
            ops.close(got[k][rows], want[k], tol[k], k)
        ops.close(got["h"][:, rows], want["h"], tol["h"], "h")


# ------------------------------------------------------------------- distillation

@pytest.mark.parametrize("T", [4, 100])
def test_loss_rows_wider_than_any_ring_with_many_entries(cuda_device, T):
    """The teacher's 1024 entries take most of half an SM's shared memory, and
    the row passes through what is left twice."""
    case = ops.loss_case(T, 300000, 1024, False, seed=T)
    got = ops.loss_run(*case, 2.0, 0.7, 0.3)
    ops.loss_check(got, ops.loss_want(*case, 2.0, 0.7, 0.3), case[4], case[0], 2.0, 0.7, 0.3)


@pytest.mark.parametrize("T,V,K,f32", [(1, 50257, 64, False), (8, 50257, 300, False), (19, 50257, 1024, False), (300, 128256, 64, False),
                                       (300, 128256, 300, False), (200, 50257, 100, True), (4, 300000, 1024, False),
                                       (3, 1000003, 130, False), (2, 16384, 20, True)])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_loss_over_the_logits_where_ctas_share_a_row(cuda_device, T, V, K, f32, tau):
    """The gradient written over the logits, by CTAs each of which reads logits
    of the others' parts for the loss: every bit as with a place of its own."""
    z, ids, teacher, labels, w = ops.loss_case(T, V, K, f32, seed=V + K)
    ids[:, K // 2] = ids[:, 1]                       # read again after the others
    ids[::2, K - 1] = ids[::2, 3]
    labels[::3] = ids[::3, 0]
    kw = dict(labels=labels, row_weight=w, temperature=tau, kd_weight=0.8, ce_weight=0.2)
    loss, stats, d = torch.empty(T, device="cuda"), torch.empty(T, 2, device="cuda"), torch.empty_like(z)
    q8.q8_distill_topk_forward(z, ids, teacher, loss, stats=stats, dlogits=d, **kw)
    d2 = torch.empty_like(z)
    q8.q8_distill_topk_backward(z, ids, teacher, stats, d2, **kw)
    for _ in range(5):
        a, b = z.clone(), z.clone()
        loss_a, stats_a = torch.empty_like(loss), torch.empty_like(stats)
        q8.q8_distill_topk_forward(a, ids, teacher, loss_a, stats=stats_a, dlogits=a, **kw)
        q8.q8_distill_topk_backward(b, ids, teacher, stats, b, **kw)
        assert torch.equal(loss_a, loss) and torch.equal(stats_a, stats) and torch.equal(a, d) and torch.equal(b, d2)
    if T <= 8:
        want = ops.loss_want(z, ids, teacher, labels, w, tau, 0.8, 0.2)
        ops.loss_check((loss, loss, loss, d, d2), want, w, z, tau, 0.8, 0.2)


def test_loss_of_labels_alone_through_autograd(cuda_device):
    z, ids, teacher, labels, w = ops.loss_case(6, 1000, 0, False, seed=3)
    want = ops.loss_want(z, ids, teacher, labels, w, 1.0, 1.0, 0.5)
    for given in ((None, None), (ids, teacher)):
        zz = z.clone().requires_grad_()
        loss = q8nn.distill_topk(zz, *given, labels=labels, ce_weight=0.5)
        d, = torch.autograd.grad((loss * w).sum(), zz)
        ops.loss_check((loss, loss, loss, d), want, w, z, 1.0, 1.0, 0.5)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [500, 60000])
def test_loss_entries_without_weight_on_masked_logits(cuda_device, V, f32):
    """A teacher's entry so far below the others that its p is 0, on a student's
    logit of -inf: it adds nothing to the loss, as an entry of -inf does."""
    z, ids, teacher, labels, w = ops.loss_case(6, V, 8, f32, seed=V)
    z[:, 300:] = -math.inf
    ids[:] = torch.arange(296, 304, device="cuda")
    teacher[:, 4:] = teacher[:, :1] - torch.tensor([1000.0, 500.0, 1e30, torch.finfo(torch.float32).max], device="cuda")
    labels[:] = 5
    none = teacher.clone()
    none[:, 4:] = -math.inf
    for tau, kd, ce in ((1.0, 1.0, 0.0), (2.0, 0.5, 0.5)):
        got = ops.loss_run(z, ids, teacher, labels, w, tau, kd, ce)
        assert torch.isfinite(got[0]).all()
        want = ops.loss_want(z, ids, none, labels, w, tau, kd, ce)
        zz = z.masked_fill(torch.isinf(z), 0.0)      # the bound's span is over the finite logits
        ops.loss_check(got, want, w, zz, tau, kd, ce)


# -------------------------------------------------------------------- block norms

@pytest.mark.parametrize("T,D", [(5, 8), (700, 64), (9, 96), (33, 264), (21, 1600), (4, 4104), (3, 97)])
@pytest.mark.parametrize("post,pre,rows", [(R.LAYER, R.RMS, 0), (R.LAYER, R.RMS, 1), (R.LAYER, R.LAYER, 0), (R.LAYER, R.NONE, 0),
                                           (R.RMS, R.RMS, 0), (R.RMS, R.LAYER, 0), (R.NONE, R.LAYER, 0)])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_without_weights_at_widths_that_threads_do_not_divide(cuda_device, T, D, post, pre, rows, f32):
    """Columns that a thread has past the row's end count in no statistic, also
    where no weight makes them zero."""
    c = ops.norm_case(T, D, post, pre, 0, rows, f32, seed=T + D)
    got = ops.norm_run(c, post, pre, T, 0.75, 1e-5)
    ops.norm_check(c, got, ops.norm_want(c, post, pre, T, 0.75, 1e-5), T, D, post, pre, T, 0.75, 1e-5)


@pytest.mark.parametrize("D", [64, 264])
def test_norm_weights_gradients_without_weights(cuda_device, D):
    """The gradients of weights and biases that are ones and zeros."""
    T = 50
    c = ops.norm_case(T, D, R.LAYER, R.RMS, 0, 0, False, seed=D)
    one = dict(c, pw=torch.ones(D, dtype=BF, device="cuda"), pb=torch.zeros(D, dtype=BF, device="cuda"),
               qw=torch.ones(D, dtype=BF, device="cuda"), qb=torch.zeros(D, dtype=BF, device="cuda"))
    want = ops.norm_want(one, R.LAYER, R.RMS, T, 1.0, 1e-5)
    got = {k: torch.empty(D, dtype=BF, device="cuda") for k in ("pw", "pb", "qw", "qb")}
    dr, dy = torch.empty_like(c["r"]), torch.empty_like(c["y"])
    q8.q8_block_norm_backward(c["r"], c["y"], c["dr"], c["dz"], dr, dy, R.LAYER, R.RMS, dpost_weight=got["pw"],
                              dpost_bias=got["pb"], dpre_weight=got["qw"], dpre_bias=got["qb"])
    out, z = torch.empty_like(c["r"]), torch.empty_like(c["y"])
    q8.q8_block_norm_forward(c["r"], c["y"], out, z, R.LAYER, R.RMS)
    ops.norm_check(one, (out, z, dict(got, r=dr, y=dy)), want, T, D, R.LAYER, R.RMS, T, 1.0, 1e-5)


def test_norm_gate_rows_without_tokens_get_zeros(cuda_device):
    """A gate's gradient is written whole: zeros where no token has the row."""
    D = 136
    c = ops.norm_case(20, D, R.RMS, R.RMS, 1, 1, False, seed=1)
    kw = dict(post_weight=c["pw"], pre_weight=c["qw"])
    gate = torch.cat([c["gate"]] * 4)
    for tokens, gate_tokens, used in ((20, 10, 2), (20, 7, 3), (20, 20, 1), (0, 5, 0), (0, None, 0)):
        r, y, dr, dz = (c[k][:tokens] for k in ("r", "y", "dr", "dz"))
        dgate, want = torch.full_like(gate, 9.0), torch.zeros_like(gate)
        q8.q8_block_norm_backward(r, y, dr, dz, None, None, R.RMS, R.RMS, gate=gate, gate_tokens=gate_tokens, dgate=dgate, **kw)
        if used:
            q8.q8_block_norm_backward(r, y, dr, dz, None, None, R.RMS, R.RMS, gate=gate[:used].contiguous(),
                                      gate_tokens=gate_tokens, dgate=want[:used], **kw)
        assert torch.equal(dgate, want), (tokens, gate_tokens)
    one = torch.full((D,), 9.0, dtype=BF, device="cuda")
    q8.q8_block_norm_backward(r, y, dr, dz, None, None, R.RMS, R.RMS, gate=c["gate"][0], dgate=one, **kw)
    assert not one.any()
    side = torch.cuda.Stream()
    one.fill_(9.0)
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        q8.q8_block_norm_backward(r, y, dr, dz, None, None, R.RMS, R.RMS, gate=c["gate"][0], dgate=one, stream=stream, **kw)
    side.synchronize()
    assert not one.any()


def test_norm_no_tokens_through_autograd(cuda_device):
    """Every parameter of the module has a gradient of zeros."""
    m = q8nn.BlockNorm(64, post="layer", pre="rms", device="cuda")
    torch.full((1 << 16,), 7.0, device="cuda")       # what the allocator gives next is not zero by chance
    r = torch.zeros(2, 0, 64, dtype=BF, device="cuda", requires_grad=True)
    out, z = m(r, torch.zeros_like(r))
    assert out.shape == z.shape == r.shape
    (out.sum() + z.sum()).backward()
    assert all(p.grad is not None and not p.grad.any() for p in m.parameters())


@pytest.mark.parametrize("T,D", [(1000, 512), (50, 97), (3, 20001)])
def test_norm_workspace_of_the_stated_size(cuda_device, T, D):
    c = ops.norm_case(T, D, R.RMS, R.RMS, 1, 1, False, seed=D)
    outs = dict(dpost_weight=torch.empty_like(c["pw"]), dgate=torch.empty_like(c["gate"]))
    a = (c["r"], c["y"], c["dr"], c["dz"], torch.empty_like(c["r"]), torch.empty_like(c["y"]), R.RMS, R.RMS)
    kw = dict(post_weight=c["pw"], pre_weight=c["qw"], gate=c["gate"], **outs)
    need = q8.q8_block_norm_workspace(*a, **kw)
    assert need > 0 and q8.q8_block_norm_workspace(c["r"][:0], c["y"][:0], None, None, None, None, R.RMS, R.RMS) == 0
    q8.q8_block_norm_backward(*a, **kw)
    want = [t.clone() for t in (a[4], a[5], *outs.values())]
    room = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    q8.q8_block_norm_backward(*a, **kw, workspace=room[:need])
    assert all(torch.equal(x, y) for x, y in zip((a[4], a[5], *outs.values()), want)) and (room[need:] == 7).all()
    with pytest.raises(q8.Q8Error, match="workspace_bytes"):
        q8.q8_block_norm_backward(*a, **kw, workspace=room[:need - 256])
    with pytest.raises(q8.Q8Error, match="post_kind"):
        q8.q8_block_norm_workspace(*a[:6], 7, R.RMS)
