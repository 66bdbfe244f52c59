"""Argument checks of the training-step operators: refused on the host, before
any launch.  No GPU is needed; the addresses are never followed."""
import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import _binding as B

NULL, SIZE, ALIGN, ARG = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from bit_blockwise_adamw_gb300 import build
    build.build()
    return q8.load_library()


def ff(**kw):
    base = dict(x=0x10000, w_gate=0x20000, w_up=0x30000, tokens=8, d_model=64, d_ff=128, x_stride=64,
                workspace=0x40000, workspace_bytes=1 << 40, act=0)
    base.update(kw)
    return B._GATED_FF.pack(*[v or 0 for v in base.values()])


FF_BAD = [(dict(x=None), NULL), (dict(w_gate=None), NULL), (dict(w_up=None), NULL), (dict(x=0x10001), ALIGN),
          (dict(tokens=-1), SIZE), (dict(tokens=1 << 30), SIZE), (dict(d_model=0), SIZE), (dict(d_ff=0), SIZE),
          (dict(d_ff=1 << 30), SIZE), (dict(x_stride=63), SIZE), (dict(act=3), ARG), (dict(act=-1), ARG)]


@pytest.mark.parametrize("kw,code", FF_BAD)
def test_ff_refuses(lib, kw, code):
    f = ff(**kw)
    assert lib.q8_gated_ff_forward(f, 0x50000, 128, None, None) == code
    assert lib.q8_gated_ff_backward(f, 0x50000, 128, None, 0x60000, 64, 0x70000, 0x80000, None) == code
    assert lib.q8_gated_ff_workspace(f, 1) == code
    assert q8.q8_last_error()


def test_ff_refuses_its_other_arguments(lib):
    f = ff()
    assert lib.q8_gated_ff_forward(None, 0x50000, 128, None, None) == NULL
    assert lib.q8_gated_ff_forward(f, None, 128, None, None) == NULL
    assert lib.q8_gated_ff_forward(f, 0x50000, 127, None, None) == SIZE
    assert lib.q8_gated_ff_forward(f, 0x50001, 128, None, None) == ALIGN
    assert lib.q8_gated_ff_forward(f, 0x50000, 128, 0x50002, None) == ALIGN
    back = lambda f, dh=0x50000, dhs=128, saved=None, dx=0x60000, dxs=64, g=0x70000, u=0x80000: \
        lib.q8_gated_ff_backward(f, dh, dhs, saved, dx, dxs, g, u, None)
    assert back(f, dh=None) == NULL
    assert back(f, dhs=1) == SIZE
    assert back(f, dxs=63) == SIZE
    assert back(f, dx=0x60001) == ALIGN
    assert back(f, g=0x70001) == ALIGN
    assert back(f, saved=0x50001) == ALIGN
    assert back(ff(workspace=None)) == NULL
    assert back(ff(workspace=0x40010)) == ALIGN
    assert back(ff(workspace_bytes=lib.q8_gated_ff_workspace(f, 1) - 1)) == SIZE
    assert lib.q8_gated_ff_workspace(f, 2) == ARG
    # nothing to do: nothing is launched
    assert lib.q8_gated_ff_forward(ff(tokens=0, x=None), None, 0, None, None) == 0
    assert back(f, dx=None, g=None, u=None) == 0


def bn(**kw):
    base = dict(residual=0x10000, y=0x20000, post_weight=0x30000, post_bias=None, pre_weight=0x40000, pre_bias=None,
                gate=0x50000, tokens=4, dim=64, gate_tokens=4, residual_stride=64, y_stride=64, post_kind=1, pre_kind=2,
                residual_dtype=0, eps=1e-5, residual_scale=1.0)
    base.update(kw)
    return B._BLOCK_NORM.pack(*[v or 0 for v in base.values()])


def grads(**kw):
    base = dict(d_residual_out=0x60000, dz=0x70000, d_residual=0x80000, d_y=0x90000, d_post_weight=0xa0000,
                d_post_bias=None, d_pre_weight=0xb0000, d_pre_bias=None, d_gate=0xc0000, d_residual_out_stride=64,
                dz_stride=64, d_residual_stride=64, d_y_stride=64, workspace=0x100000, workspace_bytes=1 << 40)
    base.update(kw)
    return B._BLOCK_NORM_GRADS.pack(*[v or 0 for v in base.values()])


@pytest.mark.parametrize("kw,code", [
    (dict(residual=None), NULL), (dict(y=None), NULL), (dict(y=0x20001), ALIGN), (dict(residual=0x10002, residual_dtype=1), ALIGN),
    (dict(post_weight=0x30001), ALIGN), (dict(gate=0x50001), ALIGN), (dict(tokens=-1), SIZE), (dict(tokens=1 << 40), SIZE),
    (dict(dim=0), SIZE), (dict(dim=32769, residual_stride=40000, y_stride=40000), SIZE), (dict(gate_tokens=0), SIZE),
    (dict(residual_stride=63), SIZE), (dict(y_stride=63), SIZE), (dict(post_kind=3), ARG), (dict(pre_kind=-1), ARG),
    (dict(residual_dtype=2), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(residual_scale=float("inf")), ARG), (dict(post_kind=0), ARG), (dict(pre_kind=0), ARG)])
def test_norm_refuses(lib, kw, code):
    n, g = bn(**kw), grads()
    assert lib.q8_block_norm_forward(n, 0x110000, 64, 0x120000, 64, None) == code
    assert lib.q8_block_norm_backward(n, g, None) == code
    assert lib.q8_block_norm_workspace(n, g) == code


@pytest.mark.parametrize("kw,code", [
    (dict(d_residual_out=0x60001), ALIGN), (dict(dz=0x70001), ALIGN), (dict(d_y=0x90001), ALIGN),
    (dict(d_pre_weight=0xb0001), ALIGN), (dict(d_y_stride=63), SIZE), (dict(d_residual_stride=1), SIZE),
    (dict(dz_stride=0), SIZE), (dict(workspace=None), NULL), (dict(workspace=0x100008), ALIGN),
    (dict(workspace_bytes=0), SIZE)])
def test_norm_backward_refuses(lib, kw, code):
    assert lib.q8_block_norm_backward(bn(), grads(**kw), None) == code


def test_norm_refuses_gradients_of_nothing(lib):
    for n in (bn(post_kind=0, post_weight=None), bn(pre_kind=0, pre_weight=None), bn(gate=None)):
        assert lib.q8_block_norm_backward(n, grads(), None) == ARG
    assert lib.q8_block_norm_forward(None, None, 0, None, 0, None) == NULL
    assert lib.q8_block_norm_backward(bn(), None, None) == NULL
    assert lib.q8_block_norm_forward(bn(), 0x110000, 63, None, 0, None) == SIZE
    assert lib.q8_block_norm_forward(bn(), None, 0, None, 0, None) == 0


def topk(**kw):
    base = dict(logits=0x10000, teacher_ids=0x20000, teacher_logits=0x30000, labels=0x40000, row_weight=0x50000, rows=4,
                vocab=100, k=8, logits_stride=100, logits_dtype=0, temperature=1.0, kd_weight=1.0, ce_weight=0.5)
    base.update(kw)
    return B._DISTILL_TOPK.pack(*[v or 0 for v in base.values()])


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), NULL), (dict(teacher_ids=None), NULL), (dict(teacher_logits=None), NULL), (dict(logits=0x10001), ALIGN),
    (dict(logits=0x10002, logits_dtype=1), ALIGN), (dict(teacher_ids=0x20004), ALIGN), (dict(labels=0x40004), ALIGN),
    (dict(teacher_logits=0x30002), ALIGN), (dict(row_weight=0x50001), ALIGN), (dict(rows=-1), SIZE), (dict(vocab=0), SIZE),
    (dict(vocab=1 << 31, logits_stride=1 << 31), SIZE), (dict(k=-1), SIZE), (dict(k=1025), SIZE), (dict(logits_stride=99), SIZE),
    (dict(logits_dtype=2), ARG), (dict(temperature=0.0), ARG), (dict(temperature=float("inf")), ARG),
    (dict(kd_weight=-0.1), ARG), (dict(ce_weight=float("nan")), ARG)])
def test_distill_refuses(lib, kw, code):
    d = topk(**kw)
    assert lib.q8_distill_topk_forward(d, 0x60000, None, None, 0, None) == code
    assert lib.q8_distill_topk_backward(d, 0x70000, 0x80000, 100, None) == code


def test_distill_refuses_its_other_arguments(lib):
    d = topk()
    assert lib.q8_distill_topk_forward(None, 0x60000, None, None, 0, None) == NULL
    assert lib.q8_distill_topk_forward(d, None, None, None, 0, None) == NULL
    assert lib.q8_distill_topk_forward(d, 0x60001, None, None, 0, None) == ALIGN
    assert lib.q8_distill_topk_forward(d, 0x60000, None, 0x80000, 99, None) == SIZE
    assert lib.q8_distill_topk_backward(d, None, 0x80000, 100, None) == NULL
    assert lib.q8_distill_topk_backward(d, 0x70000, None, 100, None) == NULL
    assert lib.q8_distill_topk_forward(topk(rows=0, logits=None), None, None, None, 0, None) == 0


def test_binding_refuses_host_tensors_and_mismatches():
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be"):
        q8.q8_gated_ff_forward(x, w, w, torch.zeros(2, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="y must be"):
        q8.q8_block_norm_forward(x, x, x, x, 1, 1)
    with pytest.raises(ValueError, match="logits must be"):
        q8.q8_distill_topk_forward(x, None, None, torch.zeros(2))
