"""The training-step operators on the GPU against plain float64 forms.

Tolerances follow from the arithmetic, not from results:
 - a bf16 output is one fp32 result rounded to nearest; bf16 has eight
   significant bits, so it is within U = 2^-8 of that result, and over many
   elements the errors' root mean square is about U / (2.3) (uniform over half a
   spacing, over the significands), below RMS = 2^-9; an fp32 accumulation of n products is within
   n * 2^-22 of the sum of their magnitudes (2^-24 for a rounded add; 2^-22
   leaves room for accumulators that truncate);
 - the operands dg and du of the feed-forward products are themselves rounded
   to bf16: U times the sum of the products' magnitudes more;
 - 2^-16 relative covers the few fp32 operations and the exponentials (each
   within a few units of 2^-23) of an element.
"""
import math

import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
import train_refs as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
RMS = 2.0 ** -9
FEW = 2.0 ** -16
ACC = 2.0 ** -22
BF = torch.bfloat16


def rnd(gen, *shape, std=1.0, mean=0.0, dtype=BF):
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def strided(t, pad, shift=0):
    """A copy of t whose rows lie `pad` elements further apart, `shift` elements into its storage."""
    big = torch.full((t.shape[0] * (t.shape[1] + pad) + shift,), 7.0, device=t.device, dtype=t.dtype)
    v = big[shift:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(t)
    return v


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %g at bound %g" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()), float(tol[bad].min() if torch.is_tensor(tol) else tol))


# ------------------------------------------------------------ gated feed-forward

def ff_case(T, D, F, seed=0, dh_std=1.0):
    g = gen(seed)
    std = D ** -0.5
    return rnd(g, T, D), rnd(g, F, D, std=std), rnd(g, F, D, std=std), rnd(g, T, F, std=dh_std)


def ff_bounds(x, wg, wu, dh, act):
    """float64 results, and the bound on each output's error."""
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    D, F, T = x.shape[1], wg.shape[0], x.shape[0]
    g = (x @ wg.T).requires_grad_()
    u = (x @ wu.T).requires_grad_()
    a = R.act(g, act)
    da, = torch.autograd.grad(a.sum(), g, create_graph=True)
    a, da, g, u = a.detach(), da.detach(), g.detach(), u.detach()
    sg, su = x.abs() @ wg.abs().T * (D * ACC), x.abs() @ wu.abs().T * (D * ACC)     # errors of g and u
    h = a * u
    eh = (U + FEW) * h.abs() + (1.2 * sg + FEW * (1 + g.abs())) * u.abs() + a.abs() * su + 1e-30
    dg, du = dh * u * da, dh * a
    # |act''| <= 1.2 for all three; act' is computed to FEW
    eg = FEW * dg.abs() + dh.abs() * (su * da.abs() + u.abs() * (1.2 * sg + FEW * (1 + g.abs())))
    eu = FEW * du.abs() + dh.abs() * (1.2 * sg + FEW * (1 + g.abs()))
    og, ou = U * dg.abs() + 1.01 * eg, U * du.abs() + 1.01 * eu              # as rounded operands
    want = dict(h=h, dx=dg @ wg + du @ wu, dwg=dg.T @ x, dwu=du.T @ x)
    ex = og @ wg.abs() + ou @ wu.abs() + 2 * F * ACC * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    exg = og.T @ x.abs() + T * ACC * (dg.abs().T @ x.abs())
    exu = ou.T @ x.abs() + T * ACC * (du.abs().T @ x.abs())
    tol = dict(h=eh, dx=ex * 1.01 + U * want["dx"].abs() + 1e-30, dwg=exg * 1.01 + U * want["dwg"].abs() + 1e-30,
               dwu=exu * 1.01 + U * want["dwu"].abs() + 1e-30)
    return want, tol


def ff_run(x, wg, wu, dh, act, save=True, **out):
    T, F = x.shape[0], wg.shape[0]
    h = out.get("h", torch.empty(T, F, dtype=BF, device="cuda"))
    saved = torch.empty(2, T, F, device="cuda") if save else None
    dx = out.get("dx", torch.empty(T, x.shape[1], dtype=BF, device="cuda"))
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    q8.q8_gated_ff_forward(x, wg, wu, h, act, saved=saved)
    q8.q8_gated_ff_backward(x, wg, wu, dh, dx, dwg, dwu, act, saved=saved)
    torch.cuda.synchronize()
    return dict(h=h, dx=dx, dwg=dwg, dwu=dwu)


# one token, few, tile edges at 128 and 256 with one beside, odd widths, long sums
FF_SIZES = [(1, 64, 64), (1, 1024, 4096), (2, 72, 136), (3, 1000, 24), (5, 33, 17), (8, 256, 1000), (9, 256, 512),
            (16, 512, 777), (17, 264, 264), (33, 100, 260), (63, 2048, 72), (64, 128, 128), (65, 136, 520),
            (127, 64, 256), (128, 512, 128), (129, 192, 384), (255, 320, 256), (256, 256, 256), (257, 257, 257),
            (300, 1, 1), (1, 1, 1), (1, 7, 3), (513, 640, 1032), (1023, 88, 2000), (40, 4104, 520), (2049, 264, 136)]


@pytest.mark.parametrize("T,D,F", FF_SIZES)
@pytest.mark.parametrize("save", [True, False])
def test_ff(cuda_device, T, D, F, save):
    act = (T + D + F) % 3
    x, wg, wu, dh = ff_case(T, D, F, seed=T + D)
    want, tol = ff_bounds(x, wg, wu, dh, act)
    got = ff_run(x, wg, wu, dh, act, save)
    for k in want:
        close(got[k], want[k], tol[k], k)
        # and the error as a whole: independent roundings of the operands (dg and
        # du, T F of each) and of the result, where there are enough of them
        rel = float((got[k].double() - want[k]).norm() / want[k].norm())
        assert rel <= (RMS if k == "h" else 1.5 * RMS) or min(got[k].numel(), T * F) < 256, (k, rel)


@pytest.mark.parametrize("act", [q8.SILU, q8.GELU_TANH, q8.GELU])
def test_ff_activations_over_their_range(cuda_device, act):
    """g from -200 to 200 with u = 1, through weights that pick out columns of x."""
    n = 128
    x = torch.zeros(n, 64, dtype=BF, device="cuda")
    x[:, 0] = torch.cat([torch.linspace(-200, 200, n // 2), torch.linspace(-6, 6, n // 2)]).to(BF)
    x[:, 1] = 1.0
    wg = torch.zeros(64, 64, dtype=BF, device="cuda")
    wu = torch.zeros(64, 64, dtype=BF, device="cuda")
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    dh = torch.ones(n, 64, dtype=BF, device="cuda")
    want, tol = ff_bounds(x, wg, wu, dh, act)
    for save in (True, False):
        got = ff_run(x, wg, wu, dh, act, save)
        for k in want:
            assert torch.isfinite(got[k]).all(), k
            close(got[k], want[k], tol[k], k)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (16, 8), (5, 3)])
@pytest.mark.parametrize("T", [1, 7, 200])
def test_ff_strides_and_alignments(cuda_device, T, pad, shift):
    D, F = 136, 272
    x, wg, wu, dh = ff_case(T, D, F, seed=9)
    want, tol = ff_bounds(x, wg, wu, dh, q8.SILU)
    out = dict(h=strided(dh, pad, shift), dx=strided(x, pad, shift))
    w = [strided(t.reshape(1, -1), 0, shift).view(F, D) for t in (wg, wu)]
    for save in (True, False):
        got = ff_run(strided(x, pad, shift), *w, strided(dh, pad, shift), q8.SILU, save, **out)
        for k in want:
            close(got[k], want[k], tol[k], k)
    if pad:                                          # nothing is written between the rows
        for t in out.values():
            assert (t.as_strided((T - 1, pad), (t.stride(0), 1), t.storage_offset() + t.shape[1]) == 7.0).all()


def test_ff_skipped_outputs_and_no_tokens(cuda_device):
    x, wg, wu, dh = ff_case(70, 64, 136, seed=4)
    want, tol = ff_bounds(x, wg, wu, dh, q8.SILU)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    q8.q8_gated_ff_backward(x, wg, wu, dh, dx, None, None)
    q8.q8_gated_ff_backward(x, wg, wu, dh, None, None, dwu)
    q8.q8_gated_ff_backward(x, wg, wu, dh, None, dwg, None)
    for k, v in dict(dx=dx, dwg=dwg, dwu=dwu).items():
        close(v, want[k], tol[k], k)
    none = x[:0]
    q8.q8_gated_ff_forward(none, wg, wu, dh[:0])
    q8.q8_gated_ff_backward(none, wg, wu, dh[:0], none, dwg, dwu)
    assert not dwg.any() and not dwu.any()


def test_ff_gradient_against_differences(cuda_device):
    """<gradient, v> against the central difference of the float64 form along v."""
    T, D, F, e = 37, 136, 200, 1e-4
    x, wg, wu, dh = ff_case(T, D, F, seed=12)
    got = ff_run(x, wg, wu, dh, q8.GELU)
    g = gen(3)
    for k, i in (("dx", 0), ("dwg", 1), ("dwu", 2)):
        args = [x.double(), wg.double(), wu.double()]
        v = got[k].double() + torch.randn(got[k].shape, generator=g, device="cuda").double() * got[k].double().std()
        side = []
        for s in (e, -e):
            a = list(args)
            a[i] = a[i] + s * v / v.norm()
            side.append((R.gated_ff(*a, q8.GELU) * dh.double()).sum())
        slope = float(side[0] - side[1]) / (2 * e)
        # bf16 results: off by about RMS of their norm, so along a unit vector by less than 4 RMS of it
        assert abs(float((got[k].double() * v).sum() / v.norm()) - slope) <= 4 * RMS * float(got[k].double().norm()), k


def test_ff_same_bits_again_and_on_another_stream(cuda_device):
    x, wg, wu, dh = ff_case(300, 520, 1032, seed=5)
    a = ff_run(x, wg, wu, dh, q8.SILU)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, saved = torch.empty_like(a["h"]), torch.empty(2, 300, 1032, device="cuda")
    dx, dwg, dwu = (torch.empty_like(a[k]) for k in ("dx", "dwg", "dwu"))
    q8.q8_gated_ff_forward(x, wg, wu, h, q8.SILU, saved=saved, stream=side)
    q8.q8_gated_ff_backward(x, wg, wu, dh, dx, dwg, dwu, q8.SILU, saved=saved, stream=side.cuda_stream)
    side.synchronize()
    for p, q in zip((h, dx, dwg, dwu), (a["h"], a["dx"], a["dwg"], a["dwu"])):
        assert torch.equal(p, q)


def test_ff_nan_stays_in_its_row(cuda_device):
    x, wg, wu, dh = ff_case(130, 64, 128, seed=6)
    x[77, 5] = float("nan")
    h = torch.empty_like(dh)
    q8.q8_gated_ff_forward(x, wg, wu, h)
    bad = torch.isnan(h).all(1)
    assert bad[77] and int(torch.isnan(h).any(1).sum()) == 1


# -------------------------------------------------------------------- block norms

def norm_case(T, D, post, pre, wb, rows, f32, seed=0):
    g = gen(seed)
    c = dict(r=rnd(g, T, D, std=2.0, dtype=torch.float32 if f32 else BF), y=rnd(g, T, D, std=0.5, mean=0.3), pw=None,
             pb=None, qw=None, qb=None, gate=None)
    if wb >= 1:
        if post:
            c["pw"] = rnd(g, D, std=0.3, mean=1.0)
        if pre:
            c["qw"] = rnd(g, D, std=0.3, mean=1.0)
    if wb >= 2:
        if post:
            c["pb"] = rnd(g, D, std=0.2)
        if pre:
            c["qb"] = rnd(g, D, std=0.2)
    if rows:
        c["gate"] = rnd(g, rows, D, std=0.4, mean=0.6)
    c["dr"] = rnd(g, T, D, dtype=c["r"].dtype)
    c["dz"] = rnd(g, T, D)
    return c


def norm_want(c, post, pre, gt, scale, eps, use=("dr", "dz")):
    d = {k: (None if v is None else v.double()) for k, v in c.items()}
    names = [k for k in ("r", "y", "pw", "pb", "qw", "qb", "gate") if d[k] is not None]
    for k in names:
        d[k].requires_grad_()
    out, z = R.block_norm(d["r"], d["y"], (post, d["pw"], d["pb"]), (pre, d["qw"], d["qb"]), d["gate"], gt, scale, eps)
    total = (out * d["dr"]).sum() * ("dr" in use) + (z * d["dz"]).sum() * ("dz" in use)
    grads = dict(zip(names, torch.autograd.grad(total, [d[k] for k in names], allow_unused=True)))
    return out.detach(), z.detach(), {k: torch.zeros_like(d[k]) if v is None else v for k, v in grads.items()}


def norm_run(c, post, pre, gt, scale, eps, use=("dr", "dz"), view=lambda t: t):
    kw = dict(post_weight=c["pw"], post_bias=c["pb"], pre_weight=c["qw"], pre_bias=c["qb"], gate=c["gate"],
              gate_tokens=gt, residual_scale=scale, eps=eps)
    r, y = view(c["r"]), view(c["y"])
    out, z = view(torch.zeros_like(c["r"])), view(torch.zeros_like(c["y"]))
    q8.q8_block_norm_forward(r, y, out, z, post, pre, **kw)
    grads = {k: (torch.zeros_like(c[k]) if c[k] is not None else None) for k in ("r", "y", "pw", "pb", "qw", "qb", "gate")}
    grads["r"], grads["y"] = view(grads["r"]), view(grads["y"])
    q8.q8_block_norm_backward(r, y, view(c["dr"]) if "dr" in use else None, view(c["dz"]) if "dz" in use else None,
                              grads["r"], grads["y"], post, pre, **kw, dpost_weight=grads["pw"], dpost_bias=grads["pb"],
                              dpre_weight=grads["qw"], dpre_bias=grads["qb"], dgate=grads["gate"])
    torch.cuda.synchronize()
    return out, z, {k: v for k, v in grads.items() if v is not None}


def norm_terms(c, post, pre, gt, scale, eps):
    """The largest term of each row's gradients of r and y, before they cancel."""
    d = {k: (None if v is None else v.double()) for k, v in c.items()}
    one = torch.ones(1, dtype=torch.float64, device="cuda")
    w = {k: one if d[k] is None else d[k].abs().max() for k in ("pw", "qw", "gate")}

    def root(v, kind):
        v = v - v.mean(1, keepdim=True) if kind == R.LAYER else v
        return one if kind == R.NONE else 1 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)

    out, _ = R.block_norm(d["r"], d["y"], (post, d["pw"], d["pb"]), (R.NONE, None, None), d["gate"], gt, scale, eps)
    dr = d["dr"].abs().amax(1, keepdim=True) + root(out, pre) * d["dz"].abs().amax(1, keepdim=True) * w["qw"]
    return dict(r=abs(scale) * dr, y=root(d["y"], post) * dr * w["gate"] * w["pw"])


def norm_check(c, got, want, T, D, post, pre, gt, scale, eps):
    """Element bounds: the forward and the rows' gradients to U (FEW in fp32)
    of the element and FEW of the row's root mean square scale (a gradient is
    what is left of terms that may cancel, wholly where dim is 1: FEW of the
    terms); the sums over
    tokens to U of the sum and FEW of the sum of magnitudes, which the root of
    the number of tokens times the largest single-element gradient bounds."""
    out, z, grads = got
    wout, wz, wgrads = want
    fine = lambda t: FEW if t.dtype == torch.float32 else U + FEW
    row = lambda w: w.square().mean(1, keepdim=True).sqrt() + w.abs().amax(1, keepdim=True) / D ** 0.5 + 1e-30
    close(out, wout, fine(out) * wout.abs() + FEW * row(wout), "r'")
    close(z, wz, fine(z) * wz.abs() + 4 * FEW * row(wz), "z")
    terms = norm_terms(c, post, pre, gt, scale, eps)
    for k in ("r", "y"):
        close(grads[k], wgrads[k], fine(grads[k]) * wgrads[k].abs() + FEW * (8 * row(wgrads[k]) + terms[k]), "d" + k)
    for k in grads:
        if k not in ("r", "y"):
            scale = wgrads[k].abs().mean() + 1e-30
            close(grads[k], wgrads[k], (U + FEW) * wgrads[k].abs() + 8 * FEW * (scale + T ** 0.5), "d" + k)


NORM_SIZES = [(1, 1), (1, 8), (1, 1024), (2, 7), (3, 64), (5, 100), (7, 129), (16, 1600), (33, 2560), (300, 96),
              (64, 4096), (9, 4097), (5, 8192), (3, 16384), (2, 32768), (2, 20001), (700, 40), (1203, 257)]


@pytest.mark.parametrize("T,D", NORM_SIZES)
@pytest.mark.parametrize("post,pre,wb,rows,f32", [
    (R.RMS, R.RMS, 1, 1, False), (R.LAYER, R.LAYER, 2, 0, True), (R.NONE, R.RMS, 1, 0, False),
    (R.LAYER, R.NONE, 2, 1, False), (R.RMS, R.LAYER, 0, -1, True), (R.NONE, R.NONE, 0, 1, False),
    (R.RMS, R.RMS, 2, 3, False)])
def test_norm(cuda_device, T, D, post, pre, wb, rows, f32):
    """rows of the gate: none, one for all, one for each token (-1), or three groups, the last one short."""
    gt = T if rows <= 1 else -(-T // rows)
    n = {0: 0, 1: 1, -1: T}.get(rows, -(-T // gt))
    gt = 1 if rows == -1 else gt
    c = norm_case(T, D, post, pre, wb, n, f32, seed=T * 7 + D)
    scale, eps = (1.0, 1e-5) if rows else (0.75, 1e-3)
    got = norm_run(c, post, pre, gt, scale, eps)
    norm_check(c, got, norm_want(c, post, pre, gt, scale, eps), T, D, post, pre, gt, scale, eps)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (16, 8), (5, 3)])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_strides_and_alignments(cuda_device, pad, shift, f32):
    T, D = 37, 264
    c = norm_case(T, D, R.RMS, R.LAYER, 2, 1, f32, seed=3)
    got = norm_run(c, R.RMS, R.LAYER, T, 1.0, 1e-5, view=lambda t: strided(t, pad, shift))
    norm_check(c, got, norm_want(c, R.RMS, R.LAYER, T, 1.0, 1e-5), T, D, R.RMS, R.LAYER, T, 1.0, 1e-5)
    if pad:
        for t in (got[0], got[1], got[2]["r"], got[2]["y"]):
            assert (t.as_strided((T - 1, pad), (t.stride(0), 1), t.storage_offset() + D) == 7.0).all()


@pytest.mark.parametrize("use", [("dr",), ("dz",), ()])
def test_norm_missing_gradients(cuda_device, use):
    T, D = 21, 200
    c = norm_case(T, D, R.LAYER, R.RMS, 2, 1, False, seed=8)
    got = norm_run(c, R.LAYER, R.RMS, T, 1.0, 1e-5, use)
    norm_check(c, got, norm_want(c, R.LAYER, R.RMS, T, 1.0, 1e-5, use), T, D, R.LAYER, R.RMS, T, 1.0, 1e-5)


def test_norm_in_place_and_partial_outputs(cuda_device):
    T, D = 50, 1000
    c = norm_case(T, D, R.RMS, R.RMS, 1, 1, False, seed=5)
    out, z, grads = norm_run(c, R.RMS, R.RMS, T, 1.0, 1e-5)
    kw = dict(post_weight=c["pw"], pre_weight=c["qw"], gate=c["gate"])
    r = c["r"].clone()
    q8.q8_block_norm_forward(r, c["y"], r, None, R.RMS, R.RMS, **kw)
    z2 = torch.empty_like(z)
    q8.q8_block_norm_forward(c["r"], c["y"], None, z2, R.RMS, R.RMS, **kw)
    assert torch.equal(r, out) and torch.equal(z, z2)
    dr, dz = c["dr"].clone(), c["dz"].clone()
    dgate = torch.empty_like(c["gate"])
    q8.q8_block_norm_backward(c["r"], c["y"], dr, dz, dr, dz, R.RMS, R.RMS, **kw)
    q8.q8_block_norm_backward(c["r"], c["y"], c["dr"], c["dz"], None, None, R.RMS, R.RMS, **kw, dgate=dgate)
    assert torch.equal(dr, grads["r"]) and torch.equal(dz, grads["y"]) and torch.equal(dgate, grads["gate"])


def test_norm_rows_of_zeros_and_no_tokens(cuda_device):
    """A row of zeros has a norm of zero (eps under the root); eps 0 gives NaN in that row alone."""
    c = norm_case(6, 64, R.RMS, R.LAYER, 1, 0, False, seed=2)
    c["r"][2], c["y"][2], c["y"][4] = 0, 0, 0
    got = norm_run(c, R.RMS, R.LAYER, 6, 1.0, 1e-5)
    norm_check(c, got, norm_want(c, R.RMS, R.LAYER, 6, 1.0, 1e-5), 6, 64, R.RMS, R.LAYER, 6, 1.0, 1e-5)
    out, z, _ = norm_run(c, R.RMS, R.LAYER, 6, 1.0, 0.0)
    assert torch.isnan(z).any(1).tolist() == [False, False, True, False, True, False]
    dw = torch.ones(64, dtype=BF, device="cuda")
    q8.q8_block_norm_forward(c["r"][:0], c["y"][:0], c["r"][:0], c["y"][:0], R.RMS, R.RMS)
    q8.q8_block_norm_backward(c["r"][:0], c["y"][:0], None, None, None, None, R.RMS, R.RMS, dpre_weight=dw)
    assert not dw.any()


def test_norm_gradient_against_differences(cuda_device):
    T, D, e = 30, 328, 1e-4
    c = norm_case(T, D, R.LAYER, R.RMS, 2, 3, True, seed=4)
    _, _, grads = norm_run(c, R.LAYER, R.RMS, 10, 0.9, 1e-5)
    g = gen(1)
    for k, gr in grads.items():
        gr = gr.double()
        v = gr + torch.randn(gr.shape, generator=g, device="cuda").double() * gr.std()
        side = []
        for s in (e, -e):
            d = {n: (None if t is None else t.double()) for n, t in c.items()}
            d[k] = d[k] + s * v / v.norm()
            out, z = R.block_norm(d["r"], d["y"], (R.LAYER, d["pw"], d["pb"]), (R.RMS, d["qw"], d["qb"]), d["gate"], 10,
                                  0.9, 1e-5)
            side.append((out * d["dr"]).sum() + (z * d["dz"]).sum())
        slope = float(side[0] - side[1]) / (2 * e)
        assert abs(float((gr * v).sum() / v.norm()) - slope) <= 4 * RMS * float(gr.norm()), k


def test_norm_same_bits_again(cuda_device):
    c = norm_case(2000, 512, R.RMS, R.RMS, 1, 1, False, seed=11)
    a = norm_run(c, R.RMS, R.RMS, 2000, 1.0, 1e-5)
    b = norm_run(c, R.RMS, R.RMS, 2000, 1.0, 1e-5)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][k], b[2][k]) for k in a[2])


# ------------------------------------------------------------------- distillation

def loss_case(T, V, K, f32, seed=0):
    g = gen(seed)
    z = rnd(g, T, V, std=3.0, dtype=torch.float32 if f32 else BF)
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(T)]) if K else \
        torch.empty(T, 0, dtype=torch.int64, device="cuda")
    teacher = torch.randn(T, ids.shape[1], generator=g, device="cuda") * 3 + 10
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    weight = torch.rand(T, generator=g, device="cuda") + 0.5
    return z, ids, teacher, labels, weight


def loss_want(z, ids, teacher, labels, weight, tau, kd, ce):
    zz = z.double().requires_grad_()
    loss = R.distill(zz, ids, teacher.double(), labels, tau, kd, ce)
    w = torch.ones_like(loss) if weight is None else weight.double()
    grad = torch.autograd.grad((loss * w).sum(), zz)[0] if loss.requires_grad else None
    return loss.detach(), torch.zeros_like(zz) if grad is None else grad


def loss_run(z, ids, teacher, labels, weight, tau, kd, ce, dlogits=None):
    """Both ways to the gradient: in the forward call, and afterwards."""
    kw = dict(labels=labels, temperature=tau, kd_weight=kd, ce_weight=ce)
    T = z.shape[0]
    loss, loss2, loss3 = (torch.full((T,), 9.0, device="cuda") for _ in range(3))
    stats = torch.empty(T, 2, device="cuda")
    d1 = torch.full_like(z, 9.0) if dlogits is None else dlogits
    d2 = torch.full_like(z, 9.0)
    q8.q8_distill_topk_forward(z, ids, teacher, loss, **kw)
    q8.q8_distill_topk_forward(z, ids, teacher, loss2, stats=stats, **kw)
    q8.q8_distill_topk_backward(z, ids, teacher, stats, d2, row_weight=weight, **kw)
    q8.q8_distill_topk_forward(z, ids, teacher, loss3, dlogits=d1, row_weight=weight, **kw)
    torch.cuda.synchronize()
    return loss, loss2, loss3, d1, d2


def loss_check(got, want, weight, z, tau, kd, ce):
    """The loss is a difference of logarithms: FEW of the logits' span over tau
    (times its factor) and of the loss.  A gradient element is a probability
    (times its factor) less another: FEW of the factor, and U of itself."""
    wloss, wgrad = want
    span = (z.double().amax(1) - z.double().amin(1)) + 30
    tol = FEW * (wloss.abs() + (kd * tau + ce) * span * 0.25) + 1e-7
    for l in got[:3]:
        close(l, wloss, tol, "loss")
    w = torch.ones_like(wloss) if weight is None else weight.double()
    fine = FEW if z.dtype == torch.float32 else U + FEW
    for d in got[3:]:
        close(d, wgrad, fine * wgrad.abs() + (FEW * w * (kd * tau + ce))[:, None] * 0.25 + 1e-30, "dlogits")


LOSS_SIZES = [(1, 1, 1), (1, 50257, 16), (2, 3, 3), (3, 100, 7), (5, 1000, 64), (4, 8191, 1), (4, 32003, 100),
              (3, 50257, 0), (2, 120000, 33), (1, 300001, 5), (200, 513, 20), (3, 4096, 1024), (9, 777, 300),
              (320, 2048, 8)]


@pytest.mark.parametrize("T,V,K", LOSS_SIZES)
@pytest.mark.parametrize("tau,kd,ce,f32", [(1.0, 1.0, 0.0, False), (2.0, 0.7, 0.3, False), (1.5, 1.0, 0.5, True),
                                           (1.0, 0.5, 0.5, False), (3.0, 0.0, 1.0, True)])
def test_loss(cuda_device, T, V, K, tau, kd, ce, f32):
    case = loss_case(T, V, K, f32, seed=T + V)
    got = loss_run(*case, tau, kd, ce)
    loss_check(got, loss_want(*case, tau, kd, ce), case[4], case[0], tau, kd, ce)


def test_loss_empty_rows_padding_and_repeats(cuda_device):
    T, V, K = 12, 333, 9
    z, ids, teacher, labels, w = loss_case(T, V, K, False, seed=77)
    ids[0] = -1                                     # no teacher
    labels[1] = -100                                # no label
    ids[2], labels[2] = -1, -100                    # neither
    ids[3, 4:] = V                                  # past the vocabulary: padding
    ids[4, 1:4] = ids[4, 0]                         # an id four times
    labels[4] = ids[4, 0]
    ids[5] = ids[5, 0]                              # nine times
    teacher[6, 2:] = -math.inf
    labels[7] = V
    ids[8, ::2] = -5
    labels[9] = ids[9, 3]
    teacher[10] = -math.inf                         # no entry has any weight
    case = (z, ids, teacher, labels, w)
    for tau, kd, ce in ((2.0, 0.6, 0.4), (1.0, 1.0, 0.0), (1.0, 0.0, 1.0)):
        got = loss_run(*case, tau, kd, ce)
        want = loss_want(*case, tau, kd, ce)
        loss_check(got, want, w, z, tau, kd, ce)
        for d in got[3:]:
            assert not d[2].any() and float(got[0][2]) == 0.0


def test_loss_masked_logits(cuda_device):
    """Logits of -inf and of the type's lowest value have probability zero; a
    teacher's entry on one makes the loss infinite, not NaN."""
    z, ids, teacher, labels, w = loss_case(6, 500, 8, False, seed=5)
    lowest = torch.finfo(BF).min
    for t, v in ((0, -math.inf), (1, lowest), (2, -math.inf)):
        z[t, 100:] = v
    ids[0] = torch.arange(8, device="cuda")
    ids[1] = torch.arange(8, device="cuda")
    ids[2] = torch.arange(96, 104, device="cuda")
    labels[:3] = 7
    teacher[2, 4:] = -math.inf                      # the masked entries have no weight: finite all the same
    z[3, 200:] = -math.inf
    ids[3] = torch.arange(196, 204, device="cuda")
    labels[3] = 0
    got = loss_run(z, ids, teacher, labels, w, 2.0, 0.5, 0.5)
    assert math.isinf(float(got[0][3])) and float(got[0][3]) > 0
    keep = [0, 1, 2, 4, 5]
    want = loss_want(z[keep], ids[keep], teacher[keep], labels[keep], w[keep], 2.0, 0.5, 0.5)
    for l in got[:3]:
        close(l[keep], want[0], FEW * (want[0].abs() + 20), "loss")
    for d in got[3:]:
        assert torch.isfinite(d).all()
        close(d[keep], want[1], (U + FEW) * want[1].abs() + FEW * 3, "dlogits")
        assert not d[0, 100:].any() and not d[1, 100:].any()


def test_loss_nan_and_all_masked_rows_stay_apart(cuda_device):
    z, ids, teacher, labels, w = loss_case(5, 2000, 4, True, seed=6)
    z[1, 55] = math.nan
    z[3] = -math.inf
    got = loss_run(z, ids, teacher, labels, w, 1.0, 1.0, 0.5)
    for l in got[:3]:
        assert torch.isnan(l).tolist() == [False, True, False, True, False]


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (16, 8), (5, 3)])
@pytest.mark.parametrize("f32", [False, True])
def test_loss_strides_alignments_and_in_place(cuda_device, pad, shift, f32):
    z, ids, teacher, labels, w = loss_case(7, 1501, 11, f32, seed=8)
    want = loss_want(z, ids, teacher, labels, w, 2.0, 0.8, 0.2)
    out = strided(z, (pad * 3) % 16, (shift + 1) % 8)
    got = loss_run(strided(z, pad, shift), ids, teacher, labels, w, 2.0, 0.8, 0.2, dlogits=out)
    loss_check(got, want, w, z, 2.0, 0.8, 0.2)
    if (pad * 3) % 16:
        gap = (pad * 3) % 16
        assert (out.as_strided((6, gap), (out.stride(0), 1), out.storage_offset() + 1501) == 7.0).all()
    kw = dict(labels=labels, row_weight=w, temperature=2.0, kd_weight=0.8, ce_weight=0.2)
    loss, stats = torch.empty(7, device="cuda"), torch.empty(7, 2, device="cuda")
    a, b = strided(z, pad, shift), strided(z, pad, shift)
    q8.q8_distill_topk_forward(a, ids, teacher, loss, dlogits=a, stats=stats, **kw)
    q8.q8_distill_topk_backward(b, ids, teacher, stats, b, **kw)
    for d in (a, b):
        loss_check((loss, loss, loss, d), want, w, z, 2.0, 0.8, 0.2)


def test_loss_gradient_against_differences(cuda_device):
    z, ids, teacher, labels, w = loss_case(6, 400, 12, True, seed=9)
    got = loss_run(z, ids, teacher, labels, w, 2.0, 0.7, 0.3)
    e = 1e-4
    for d in got[3:]:
        v = torch.randn(z.shape, generator=gen(2), device="cuda").double() * d.double().std() + d.double()
        side = [(R.distill(z.double() + s * v / v.norm(), ids, teacher.double(), labels, 2.0, 0.7, 0.3) *
                 w.double()).sum() for s in (e, -e)]
        slope = float(side[0] - side[1]) / (2 * e)
        assert abs(float((d.double() * v).sum() / v.norm()) - slope) <= 4 * FEW * float(d.double().norm()) + 1e-6


def test_loss_without_labels_weights_or_teacher(cuda_device):
    z, ids, teacher, labels, w = loss_case(4, 900, 6, False, seed=10)
    got = loss_run(z, ids, teacher, None, None, 1.0, 1.0, 1.0)
    loss_check(got, loss_want(z, ids, teacher, None, None, 1.0, 1.0, 1.0), None, z, 1.0, 1.0, 1.0)
    got = loss_run(z, None, None, labels, w, 1.0, 1.0, 1.0)
    loss_check(got, loss_want(z, ids[:, :0], teacher[:, :0], labels, w, 1.0, 1.0, 1.0), w, z, 1.0, 1.0, 1.0)
    empty = torch.empty(0, device="cuda")
    q8.q8_distill_topk_forward(z[:0], ids[:0], teacher[:0], empty)


# ------------------------------------------------- offsets that pass 32 bits

def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 elements to a matrix: the last rows against the same rows alone."""
    last = 40

    T, V = 42800, 50257
    z = torch.empty(T, V, dtype=BF, device="cuda").normal_(0, 2, generator=gen(1))
    tail, ids, teacher, labels, w = loss_case(last, V, 9, False, seed=2)
    z[-last:] = tail
    all_ids = ids[torch.arange(T, device="cuda") % last]
    all_ids[-last:] = ids
    spread = lambda t: torch.cat([t[torch.arange(T - last, device="cuda") % last], t])
    loss = torch.empty(T, device="cuda")
    q8.q8_distill_topk_forward(z, all_ids, spread(teacher), loss, dlogits=z, labels=spread(labels), row_weight=spread(w),
                               temperature=2.0, kd_weight=0.5, ce_weight=0.5)
    got = (loss[-last:],) * 3 + (z[-last:],)
    loss_check(got, loss_want(tail, ids, teacher, labels, w, 2.0, 0.5, 0.5), w, tail, 2.0, 0.5, 0.5)
    del z, loss

    T, D = 540000, 4096
    c = norm_case(last, D, R.RMS, R.LAYER, 1, 0, False, seed=3)
    big = {k: torch.empty(T, D, dtype=BF, device="cuda").normal_(0, 1, generator=gen(4)) for k in ("r", "y", "dr", "dz")}
    for k, t in big.items():
        t[-last:] = c[k]
    kw = dict(post_weight=c["pw"], pre_weight=c["qw"])
    q8.q8_block_norm_backward(big["r"], big["y"], big["dr"], big["dz"], big["dr"], big["dz"], R.RMS, R.LAYER, **kw)
    z = torch.empty_like(big["y"])
    q8.q8_block_norm_forward(big["r"], big["y"], big["r"], z, R.RMS, R.LAYER, **kw)
    got = (big["r"][-last:], z[-last:], dict(r=big["dr"][-last:], y=big["dz"][-last:]))
    want = norm_want(c, R.RMS, R.LAYER, last, 1.0, 1e-5)
    norm_check(c, got, want, last, D, R.RMS, R.LAYER, last, 1.0, 1e-5)
    del big, z

    T, D, F = 135000, 64, 16384
    x, wg, wu, dh = ff_case(T, D, F, seed=5)
    got = ff_run(x, wg, wu, dh, q8.SILU, save=False)
    want, tol = ff_bounds(x[-last:], wg, wu, dh[-last:], q8.SILU)
    for k in ("h", "dx"):
        close(got[k][-last:], want[k], tol[k], k)
