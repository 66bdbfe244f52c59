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
