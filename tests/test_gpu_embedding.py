"""The token embedding and its gradient on the GPU, against float64.

Tolerances.  u is half a step of the result's type (bf16 2^-8, float32 2^-24).
Lookup: the product is rounded to float32 and then to the type.  Gradient: a sum
of n float32 terms is off by at most (n - 1) 2^-24 sum|d| in any association (to
first order; the second is below a hundredth of it for n up to 2^18), the
product with the scale or the addition to what is there by 2^-24 of the result,
and the result by u.  The smallest steps of the types are added throughout."""
import os
import subprocess
import sys

import pytest
import torch

import bit_blockwise_adamw_gb300 as q8

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -133, F32: 2.0 ** -149}


def rnd(*shape, seed=0, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def make_ids(kind, T, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 5)
    R = lambda lo, hi: torch.randint(lo, hi, (T,), generator=g, device="cuda")
    if kind == "uniform":
        return R(0, V)
    if kind == "one":                               # all tokens alike
        return torch.full((T,), V // 2, device="cuda")
    if kind == "skewed":                            # as words fall off
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        return ((V + 1.0) ** u - 1).long().clamp(0, V - 1)
    if kind == "padded":                            # half of them one token, some none at all
        ids = R(0, V)
        ids[torch.rand(T, generator=g, device="cuda") < 0.5] = V - 1
        ids[torch.rand(T, generator=g, device="cuda") < 0.1] = -100
        return ids
    if kind == "outside":                           # none of them in the table, at every distance
        far = torch.tensor([-1, V, V + 1, -100, 1 << 31, 1 << 32, (1 << 62) + 1, -(1 << 63), (1 << 32) + V // 2], device="cuda")
        return far[R(0, len(far))]
    if kind == "ends":                              # the first and the last row, and just past them
        return torch.tensor([0, V - 1, -1, V], device="cuda")[R(0, 4)]
    if kind == "runs":                              # sorted, each id a few times
        return (torch.arange(T, device="cuda") // 3) % V
    raise KeyError(kind)


def strided(rows, cols, dtype, extra, offset, fill=0.0):
    """A [rows, cols] matrix whose rows are `extra` elements apart, `offset` elements into its memory, and that memory."""
    buf = torch.full((offset + max(rows, 1) * (cols + extra) + 64,), fill, dtype=dtype, device="cuda")
    return buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols], buf


def check_lookup(ids, table, out, scale):
    V = table.shape[0]
    known = (ids >= 0) & (ids < V)
    want = torch.where(known[:, None], table.double()[ids.clamp(0, V - 1)] * scale, 0.0)
    off = (out.double() - want).abs()
    u = U[out.dtype]
    assert bool((off <= want.abs() * ((1 + 2.0 ** -24) * (1 + u) - 1) + TINY[out.dtype]).all()), float(off.max())


def check_grad(ids, dout, got, scale, base=None):
    V, D = got.shape
    known = (ids >= 0) & (ids < V)
    at = ids[known]
    # where a row's sum is of many terms, float64's own error is 2^-29 of float32's
    total = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, at, dout[known].double())
    size = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, at, dout[known].double().abs())
    n = torch.bincount(at, minlength=V).double()[:, None]
    want = total * scale
    if base is not None:
        want = want + base.double()
    allowed = 1.01 * abs(scale) * size * (n - 1).clamp(min=0) * 2.0 ** -24
    allowed = (want.abs() + allowed) * ((1 + 2.0 ** -24) * (1 + U[BF]) - 1) + allowed + TINY[BF]
    off = (got.double() - want).abs()
    assert bool((off <= allowed).all()), float((off / allowed).max())
    absent = n[:, 0] == 0
    if base is None:
        assert bool((got[absent].view(torch.int16) == 0).all()), "rows without a token"
    else:
        assert torch.equal(got[absent], base[absent])


SIZES = [(1, 1, 1), (1, 50257, 64), (255, 3, 257), (256, 40, 24), (256, 5000, 1031), (3, 7, 8), (33, 10, 5), (257, 1000, 136), (300, 513, 264), (1000, 65537, 33), (2049, 300, 96),
         (5000, 70000, 40), (777, 2000, 1601), (130, 999, 4104), (19, 64, 9000),
         (257, 50257, 712), (1500, 50257, 1000), (4096, 900, 24), (4097, 900, 24), (8193, 40, 520), (32769, 300, 8)]
KINDS = ["uniform", "one", "skewed", "padded", "outside", "ends", "runs"]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_lookup(cuda_device, T, V, D, dtype):
    table = rnd(V, D, seed=1)
    for i, kind in enumerate(KINDS):
        ids = make_ids(kind, T, V, seed=i)
        out = torch.full((T, D), float("nan"), dtype=dtype, device="cuda")
        scale = (1.0, 0.3, -64.0)[i % 3]
        q8.q8_embedding_forward(ids, table, out, scale=scale)
        check_lookup(ids, table, out, scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_gradient(cuda_device, T, V, D, dtype):
    dout = rnd(T, D, seed=2, dtype=dtype)
    base = rnd(V, D, seed=3)
    for i, kind in enumerate(KINDS):
        ids = make_ids(kind, T, V, seed=10 + i)
        scale = (1.0, 0.3, -64.0)[i % 3]
        got = torch.full((V, D), float("nan"), dtype=BF, device="cuda")
        q8.q8_embedding_backward(ids, dout, got, scale=scale)
        check_grad(ids, dout, got, scale)
        again = torch.full_like(got, 3.0)
        q8.q8_embedding_backward(ids, dout, again, scale=scale)
        assert torch.equal(got.view(torch.int16), again.view(torch.int16)), "the same call gives the same bits"
        got = base.clone()
        q8.q8_embedding_backward(ids, dout, got, scale=scale, accumulate=True)
        check_grad(ids, dout, got, scale, base)


@pytest.mark.parametrize("T,V,D", [(6000, 5000, 264), (40000, 50257, 72), (70000, 130000, 24), (262144, 50257, 8), (300001, 17, 16),
                                   (1300001, 50257, 8)])
@pytest.mark.parametrize("kind", ["uniform", "one", "skewed", "padded"])
def test_gradient_of_many_tokens_is_exact_on_whole_numbers(cuda_device, T, V, D, kind):
    """Sums of small whole numbers are exact in float32 in any order (below
    2^24): the result has to be their one rounding, however many tokens."""
    ids = make_ids(kind, T, V, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T)
    dout = torch.randint(-8, 9, (T, D), generator=g, device="cuda").to(BF)
    got = torch.full((V, D), float("nan"), dtype=BF, device="cuda")
    q8.q8_embedding_backward(ids, dout, got, scale=0.5)
    known = (ids >= 0) & (ids < V)
    total = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids[known], dout[known].double())
    assert float(total.abs().max()) < 2 ** 24
    assert torch.equal(got, (total * 0.5).float().to(BF))


def test_tens_of_millions_of_tokens(cuda_device):
    """More rows than a launch has CTAs, more tokens than the sort's CTAs hold at
    once; whole numbers, so that every result is known exactly."""
    T, V, D = 34000001, 1000, 9
    ids = make_ids("padded", T, V, seed=3)
    ids[:T // 2] = make_ids("uniform", T // 2, V, seed=4)
    table = torch.randint(-100, 101, (V, D), device="cuda").to(BF)
    out = torch.empty(T, D, dtype=BF, device="cuda")
    q8.q8_embedding_forward(ids, table, out, scale=-1.0)
    for t in torch.arange(T, device="cuda").split(1 << 22):
        known = (ids[t] >= 0) & (ids[t] < V)
        assert torch.equal(out[t], torch.where(known[:, None], -table[ids[t].clamp(0, V - 1)], 0.0).to(BF) + 0.0)
    out.view(torch.int16).random_(0, 2)              # ones and zeros, as bits
    out = out.view(torch.int16).to(BF)
    got = torch.full((V, D), float("nan"), dtype=BF, device="cuda")
    q8.q8_embedding_backward(ids, out, got)
    total = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    for t in torch.arange(T, device="cuda").split(1 << 22):
        known = t[(ids[t] >= 0) & (ids[t] < V)]
        total.index_add_(0, ids[known], out[known].double())
    assert float(total.max()) < 2 ** 24 and torch.equal(got, total.float().to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,extra,offset", [(64, 0, 1), (64, 3, 0), (64, 8, 8), (61, 0, 0), (61, 3, 5), (264, 8, 4), (1600, 1, 0), (2056, 8, 0)])
def test_strides_and_alignment(cuda_device, dtype, D, extra, offset):
    T, V = 515, 200
    ids = make_ids("padded", T, V, seed=4)
    for toff in (0, 1):
        tbuf = rnd(V * D + 8, seed=5)
        table = tbuf[toff:toff + V * D].view(V, D)
        out, buf = strided(T, D, dtype, extra, offset, fill=7.0)
        q8.q8_embedding_forward(ids, table, out, scale=0.7)
        check_lookup(ids, table, out, 0.7)
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[offset:offset + T * (D + extra)].view(T, D + extra)[:, :D] = False
        assert bool((buf[rest] == 7.0).all()), "memory between and behind the rows"
        dout, _ = strided(T, D, dtype, extra, offset, fill=float("nan"))
        dout.copy_(rnd(T, D, seed=6, dtype=dtype))
        gbuf = torch.full((V * D + 16,), 7.0, dtype=BF, device="cuda")
        got = gbuf[toff:toff + V * D].view(V, D)
        q8.q8_embedding_backward(ids, dout, got, scale=0.7)
        check_grad(ids, dout, got, 0.7)
        assert bool((gbuf[:toff] == 7.0).all()) and bool((gbuf[toff + V * D:] == 7.0).all())


def test_rows_of_no_token_are_not_read(cuda_device):
    """NaN and infinities in dout's rows without a token, in the table's rows
    that no token has, and behind the last token, reach nothing."""
    T, V, D = 100, 50, 72
    ids = make_ids("uniform", T, V // 2)
    ids[::3] = -1
    table = rnd(V, D)
    table[V // 2:] = float("nan")
    out = torch.empty(T, D, dtype=BF, device="cuda")
    q8.q8_embedding_forward(ids, table, out)
    assert bool(out.isfinite().all()) and bool((out[::3] == 0).all())
    dout = rnd(T + 5, D)
    dout[:T:3] = float("nan")
    dout[T:] = float("inf")
    got = torch.empty(V, D, dtype=BF, device="cuda")
    q8.q8_embedding_backward(ids, dout[:T], got)
    assert bool(got.isfinite().all())
    got = torch.full((V, D), float("nan"), dtype=BF, device="cuda")
    q8.q8_embedding_backward(ids, dout[:T], got, accumulate=True)
    assert bool(got.isnan().all()), "what is there is added to"
    dout[1] = float("inf")                          # and one row with a token does
    q8.q8_embedding_backward(ids, dout[:T], got)
    assert bool(got[ids[1]].isinf().all()) and int((~got.isfinite()).any(1).sum()) == 1


def test_no_tokens(cuda_device):
    ids, empty = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda")
    table = rnd(9, 24)
    q8.q8_embedding_forward(ids, table, empty)
    got = table.clone()
    q8.q8_embedding_backward(ids, empty, got, accumulate=True)
    assert torch.equal(got, table)
    q8.q8_embedding_backward(ids, empty, got)
    assert not got.any()


def test_the_gradient_is_the_lookups_by_differences(cuda_device):
    """sum(dout * lookup(W)) is linear in W: its difference over a step h in one
    element is h * dW there.  Whole numbers and powers of two keep all of it exact."""
    T, V, D = 60, 20, 16
    ids = make_ids("skewed", T, V, seed=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    table, dout = (torch.randint(-4, 5, s, generator=g, device="cuda").to(BF) for s in ((V, D), (T, D)))
    dw = torch.empty(V, D, dtype=BF, device="cuda")
    q8.q8_embedding_backward(ids, dout, dw, scale=2.0)
    value = lambda w: (lookup(ids, w, 2.0).double() * dout.double()).sum()

    def lookup(ids, w, scale):
        out = torch.empty(T, D, dtype=F32, device="cuda")
        q8.q8_embedding_forward(ids, w, out, scale=scale)
        return out
    for v, c in ((0, 0), (1, 5), (V - 1, D - 1), (3, 7)):
        w = table.clone()
        w[v, c] += 1
        assert float(value(w) - value(table)) == float(dw[v, c])


def test_offsets_past_32_bits(cuda_device):
    """A table and rows of more than 2^31 elements each (2^32 bytes and more)."""
    V, D, T = 270000, 8192, 300
    table = torch.empty(V, D, dtype=BF, device="cuda")
    table.view(torch.int16).random_(0, 0x3F80)
    ids = make_ids("uniform", T, V)
    ids[:4] = torch.tensor([0, V - 1, 262144, V - 2], device="cuda")
    out = torch.empty(T, D, dtype=F32, device="cuda")
    q8.q8_embedding_forward(ids, table, out)
    assert torch.equal(out, table[ids].float())
    dout = rnd(T, D)
    q8.q8_embedding_backward(ids, dout, table)                  # the table's memory serves as the gradient's
    for v in ids.unique().tolist():
        assert torch.equal(table[v], dout[ids == v].float().sum(0).to(BF)) or int((ids == v).sum()) > 2
    present = torch.zeros(V, dtype=torch.bool, device="cuda")
    present[ids] = True
    for rows in torch.arange(V, device="cuda").split(30000):
        assert bool((table[rows][~present[rows]] == 0).all())
    del table, out, dout
    T, V, D = 540000, 100, 4096
    wide = torch.zeros(T, D, dtype=BF, device="cuda")
    wide[-1], wide[0], wide[T - 7] = 1.0, 2.0, 4.0
    ids = torch.zeros(T, dtype=torch.int64, device="cuda")
    ids[-1], ids[T - 7] = 99, 98
    got = torch.empty(V, D, dtype=BF, device="cuda")
    q8.q8_embedding_backward(ids, wide, got)
    assert bool((got[99] == 1).all()) and bool((got[98] == 4).all()) and bool((got[0] == 2).all()) and not got[1:98].any()
    ids.fill_(99)
    q8.q8_embedding_forward(ids, got, wide)
    assert bool((wide[-1] == 1).all()) and bool((wide[T // 2:] == 1).all())


def test_other_streams_and_workspaces(cuda_device):
    """Calls on two streams at once, one with a workspace of the caller's."""
    T, V, D = 9000, 5000, 264
    a, b = (make_ids("skewed", T, V, seed=i) for i in (1, 2))
    dout = rnd(T, D)
    want = [torch.empty(V, D, dtype=BF, device="cuda") for _ in "ab"]
    for ids, w in zip((a, b), want):
        q8.q8_embedding_backward(ids, dout, w)
    ws = torch.empty(max(1, q8.q8_embedding_workspace(b, dout, want[1])), dtype=torch.uint8, device="cuda").random_(0, 255)
    got = [torch.full_like(w, 9.0) for w in want]
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(one):
            q8.q8_embedding_backward(a, dout, got[0])
        q8.q8_embedding_backward(b, dout, got[1], workspace=ws, stream=two)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.int16), w.view(torch.int16))


CHILD = r"""
import torch
import bit_blockwise_adamw_gb300 as q8
q8.q8_prepare_device()
BF = torch.bfloat16
g = torch.Generator(device="cuda").manual_seed(1)
E = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")
for T, V, D, dt in ((1, 500, 64, BF), (3000, 50257, 136, BF), (20000, 3000, 61, torch.float32)):
    ids = torch.randint(-2, V + 2, (T,), generator=g, device="cuda")
    table, dout = torch.randn(V, D, device="cuda").to(BF), torch.randn(T, D, device="cuda").to(dt)
    def calls(o):
        q8.q8_embedding_forward(ids, table, o[0], scale=3.0)
        q8.q8_embedding_backward(ids, dout, o[1], scale=3.0)
        q8.q8_embedding_backward(ids, dout, o[2], accumulate=True)
    new = lambda: (E(T, D, dtype=dt), E(V, D), torch.ones(V, D, dtype=BF, device="cuda"))
    a, b = new(), new()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(a)
    for other in (False, True):                      # replayed, and replayed on other inputs
        if other:
            ids.copy_(torch.randint(0, V, (T,), generator=g, device="cuda"))
            dout.mul_(-0.5)
        for o in (a, b):
            o[2].fill_(1.0)
        graph.replay()
        calls(b)
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (T, V, D, other)
print("OK")
"""


def test_captured_in_a_graph_after_prepare(cuda_device):
    env = dict(os.environ)
    env["PYTHONPATH"] = os.pathsep.join([ROOT, env.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
