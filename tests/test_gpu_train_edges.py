"""Edges of the training-step operators on the GPU: sizes and calls at which a
launch takes another shape, against the float64 forms and within the bounds of
test_gpu_train_ops."""
import pytest
import torch

import bit_blockwise_adamw_gb300 as q8
import test_gpu_train_ops as ops

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


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
