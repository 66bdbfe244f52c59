"""The embedding's gradient at the borders of its sorts and of its narrowest rows,
on whole numbers: every sum is exact in float32, and its one rounding is known."""
import pytest
import torch

import bit_blockwise_adamw_gb300 as q8

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def whole(T, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-8, 9, (T, D), generator=g, device="cuda").to(dtype)


def ids_of(T, V, seed):
    """A third of them in the last rows, a few frequent ones, some outside the table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(-2, V + 2, (T,), generator=g, device="cuda")
    u = torch.rand(T, generator=g, device="cuda")
    ids = torch.where(u < 0.3, V - 1 - ids % min(V, 100), ids)
    return torch.where(u > 0.8, ids % min(V, 3), ids)


def check(ids, dout, V, out=None):
    D = dout.shape[1]
    known = (ids >= 0) & (ids < V)
    total = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids[known], dout[known].double())
    got = torch.full((V, D), float("nan"), dtype=BF, device="cuda") if out is None else out
    q8.q8_embedding_backward(ids, dout, got, scale=0.5)
    assert torch.equal(got, (total * 0.5).float().to(BF))
    got.fill_(3.0)
    q8.q8_embedding_backward(ids, dout, got, scale=0.5, accumulate=True)
    assert torch.equal(got, (total * 0.5 + 3.0).float().to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 2, 3])
@pytest.mark.parametrize("T", [300, 5000, 40000])
def test_narrow_rows_at_every_alignment(cuda_device, T, D, dtype):
    """Rows of a column or two, of which one 32-bit word holds several: what lies
    before the first row and behind the last one reaches nothing."""
    V = 700
    ids = ids_of(T, V, seed=T + D)
    ids[0], ids[-2:] = 5, torch.tensor([7, 9], device="cuda")
    rows = whole(T, D, dtype, seed=D)
    for extra in (0, 1, 2):
        for at in (0, 1, 2, 3):
            buf = torch.full((T * (D + extra) + 8,), float("nan"), dtype=dtype, device="cuda")
            dout = buf[at:at + T * (D + extra)].view(T, D + extra)[:, :D]
            dout.copy_(rows)
            table = torch.full((V * D + 8,), float("nan"), dtype=BF, device="cuda")
            check(ids, dout, V, table[at:at + V * D].view(V, D))
            assert bool(table[:at].isnan().all()) and bool(table[at + V * D:].isnan().all())


@pytest.mark.parametrize("T", [300, 5000, 32768, 32769, 100003])
@pytest.mark.parametrize("V,D", [((1 << 18) - 1, 8), (1 << 18, 8), ((1 << 18) + 1, 3), ((1 << 27) - 1, 1), (1 << 27, 1)])
def test_vocabularies_at_the_borders_of_the_sorts_passes(cuda_device, T, V, D):
    """Nine bits a pass, the key of ids outside the table among them: two passes
    to vocabularies of 2^18 - 1, three to 2^27 - 1, then four; sorted by
    comparison, by one cluster and by all SMs."""
    check(ids_of(T, V, seed=T), whole(T, D, BF, seed=T), V)
