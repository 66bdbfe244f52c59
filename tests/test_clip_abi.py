"""Lists that clipping refuses because one entry's output is another's gradient or
output: refused on the host, before any launch.  No GPU is needed; the addresses
are never followed: what passes the check is refused for its max_norm."""
import random

import pytest

import bit_blockwise_adamw_gb300 as q8
from bit_blockwise_adamw_gb300 import _binding as B

ARG = -4
BF, F32 = 0, 1


@pytest.fixture(scope="module")
def refused():
    """The entry that clipping refuses for what it overlaps, or None."""
    from bit_blockwise_adamw_gb300 import build
    build.build()
    lib = q8.load_library()

    def call(entries):
        entries = [e if len(e) == 5 else (*e, BF, BF) for e in entries]
        data = b"".join(B._GRAD.pack(*e) for e in entries)
        assert lib.q8_clip_grads(data, len(entries), -1.0, 0x30000, 0x40000, 1 << 40, None) == ARG
        said = q8.q8_last_error()
        assert "overlap" in said or "max_norm" in said
        return int(said.split("gradient ")[-1].rstrip(")")) if "overlap" in said else None
    return call


def test_entries_apart_are_taken(refused):
    assert refused([(0x1000, 0x1000, 8), (0x1010, 0x1010, 8), (0x2000, 0x2000, 100)]) is None
    assert refused([(0x2000, 0x2000, 100), (0x1010, 0x1010, 8), (0x1000, 0x1000, 8)]) is None
    assert refused([(0x1000, 0x8000, 8), (0x1000, 0x8010, 8)]) is None        # one gradient, to two places
    assert refused([(0x1000, 0x1010, 8), (0x1020, 0x1030, 8)]) is None        # gradients and outputs in turn
    assert refused([(0x1000, 0x1000, 8), (0x1000, 0x1000, 0), (0, 0, 0)]) is None
    assert refused([(0x1000, 0x1000, 4, F32, F32), (0x1010, 0x1010, 8)]) is None


@pytest.mark.parametrize("entries,at", [
    ([(0x1000, 0x1000, 8), (0x1000, 0x1000, 8)], 1),                          # the same tensor twice
    ([(0x1000, 0x1000, 8), (0x2000, 0x2000, 8), (0x1000, 0x1000, 8)], 2),
    ([(0x1000, 0x1000, 9), (0x1010, 0x1010, 8)], 1),                          # one element of two tensors
    ([(0x1010, 0x1010, 8), (0x1000, 0x1000, 9)], 0),
    ([(0x1000, 0x1000, 5, F32, F32), (0x1010, 0x1010, 8)], 1),
    ([(0x1000, 0x8000, 8), (0x2000, 0x8000, 8)], 1),                          # two gradients to one place
    ([(0x1000, 0x8000, 8), (0x2000, 0x800e, 8)], 1),
    ([(0x1000, 0x2000, 8), (0x2000, 0x8000, 8)], 1),                          # an output over another's gradient
    ([(0x1000, 0x8000, 8), (0x2000, 0x100e, 8)], 0),
    ([(0x1000, 0x1002, 8)], 0),                                               # and over its own, shifted
    ([(0x1000, 0x1010, 8, BF, F32), (0x102e, 0x8000, 1)], 1)])
def test_overlapping_entries_are_refused(refused, entries, at):
    assert refused(entries) == at


def test_against_all_pairs(refused):
    rng = random.Random(1)
    seen = set()
    for _ in range(600):
        entries = []
        for _ in range(rng.randint(1, 6)):
            gd, od, n = rng.choice((BF, F32)), rng.choice((BF, F32)), rng.randint(0, 12)
            g = rng.randrange(0x1000, 0x1300, 4)
            o = g if rng.random() < 0.5 and gd == od else rng.randrange(0x1000, 0x1300, 4)
            if o != g or gd == od:
                entries.append((g, o, n, gd, od))
        entries = entries or [(0x1000, 0x1000, 1, BF, BF)]
        span = lambda p, n, d: range(p, p + n * (4 if d == F32 else 2))
        meet = lambda a, b: len(a) > 0 and len(b) > 0 and a[0] < b[-1] + 1 and b[0] < a[-1] + 1
        bad = False
        for i, (g, o, n, gd, od) in enumerate(entries):
            for j, (h, p, m, hd, pd) in enumerate(entries):
                bad |= i != j and (meet(span(o, n, od), span(p, m, pd)) or meet(span(o, n, od), span(h, m, hd)))
            bad |= g != o and meet(span(g, n, gd), span(o, n, od))
        assert (refused(entries) is not None) == bad, entries
        seen.add(bad)
    assert seen == {True, False}


def test_the_norm_alone_takes_a_gradient_twice():
    data = B._GRAD.pack(0x1000, 0x1000, 8, BF, BF) * 2
    assert q8.load_library().q8_grad_norm(data, 2, None, 0x40000, 1 << 40, None) == -1
    assert "norm is NULL" in q8.q8_last_error()
