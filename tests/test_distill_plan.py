"""The launch shapes of the distillation kernel (csrc/q8_distill_plan.h), walked
over the documented ranges on the host: every one has a ring its rows can go
through, within an SM's shared memory."""
import ctypes as C
import os
import random
import subprocess

import pytest

from bit_blockwise_adamw_gb300 import _binding as B
from bit_blockwise_adamw_gb300 import build

FORWARD, TRAIN, STREAM = 0, 1, 2                    # Mode
FIFTH, HALF, WHOLE = 0, 1, 2                        # Shape
SLOTS, CTA, SM = 16, 227 * 1024, 228 * 1024         # ring's most slots; shared memory of a CTA at most, of an SM

SOURCE = r"""
#include "q8_distill_plan.h"
extern "C" void plan(const void* d, int grad, int first_pass, int sms, int64_t out[10])
{
    using namespace q8::distill;
    const Config c = configure(*static_cast<const q8_distill_topk*>(d), grad != 0, first_pass != 0, sms);
    const int64_t v[10] = {c.mode, c.ctas, c.shape, c.slots, c.chunk, c.seen, static_cast<int64_t>(c.smem), threads_of(c.shape), ctas_per_sm(c.shape), c.usable};
    for (int i = 0; i < 10; ++i) out[i] = v[i];
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = str(d / "plan.cpp"), str(d / "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", build.INCLUDE, "-I", build.CSRC, src,
                    "-o", so], check=True)
    lib = C.CDLL(so)
    lib.plan.argtypes = [C.c_char_p, C.c_int, C.c_int, C.c_int, C.POINTER(C.c_int64)]
    lib.plan.restype = None
    out = (C.c_int64 * 10)()

    def call(rows, vocab, k, f32, grad, first_pass, sms=152):
        d = B._DISTILL_TOPK.pack(0, 0, 0, 0, 0, rows, vocab, k, vocab, int(f32), 1.0, 1.0, 1.0)
        lib.plan(d, int(grad), int(first_pass), sms, out)
        return dict(zip(("mode", "ctas", "shape", "slots", "chunk", "seen", "smem", "threads", "per_sm", "usable"), out))
    return call


def sound(p, vocab, k, f32, grad, first_pass):
    """The ring takes a CTA's slice of the row; what the kernel keeps of the
    teacher and the ring fit together; and an SM holds as many CTAs as meant."""
    vectors = max(1, vocab * (4 if f32 else 2) // 16)
    share = -(-vectors // p["ctas"])
    chunks = -(-share // p["chunk"]) if p["chunk"] > 0 else None
    entries = (k + 4) // 4 * 4
    teacher = entries * (3 * 16 + 2 * 12) + 4 * p["seen"]        # three rows prepared, two as they come, the ids' table
    modes = (FORWARD,) if not grad else (TRAIN, STREAM) if first_pass else (STREAM,)
    return (p["usable"] == 1 and p["mode"] in modes and p["ctas"] in (1, 2, 4, 8) and 1 <= p["chunk"] <= share
            and 2 <= p["slots"] <= SLOTS and (p["mode"] != TRAIN or p["slots"] >= chunks + 3)
            and p["seen"] >= 2 * k and p["seen"] & (p["seen"] - 1) == 0
            and p["slots"] * p["chunk"] * 16 + teacher == p["smem"]
            and p["smem"] + 1536 <= CTA and (p["smem"] + 1536 + 1024) * p["per_sm"] <= SM)


WAYS = [(False, True), (True, True), (True, False)]              # gradient, first pass: forward, both, gradient from statistics


def test_every_size_has_a_ring(plan):
    rng = random.Random(1)
    vocabs = {1, 2, 7, 8, 9, 500, 1024, 4095, 4096, 8191, 8192, 16384, 32003, 50257, 73000, 128256, 294900, 294920, 300000, 393216,
              400001, 1000003, 1 << 24, (1 << 31) - 1}
    vocabs |= {int(round(2 ** rng.uniform(0, 31))) - 1 or 1 for _ in range(120)}
    ks = {0, 1, 3, 4, 63, 64, 65, 127, 128, 129, 300, 500, 555, 560, 575, 600, 767, 1000, 1008, 1011, 1012, 1015, 1016, 1020, 1023, 1024}
    bad = []
    for vocab in sorted(vocabs):
        for k in ks:
            for f32 in (False, True):
                for grad, first in WAYS:
                    for rows in (1, 4, 9, 10, 19, 20, 38, 76, 77, 8192):
                        p = plan(rows, vocab, k, f32, grad, first)
                        if not sound(p, vocab, k, f32, grad, first):
                            bad.append((rows, vocab, k, f32, grad, first, p))
    assert not bad, "%d of the sizes, the first %r" % (len(bad), bad[0])


@pytest.mark.parametrize("rows", [1, 4, 8192])
@pytest.mark.parametrize("k", [1016, 1024])
def test_wide_rows_with_many_entries(plan, rows, k):
    """Rows that no cluster's shared memory holds, beside a teacher that takes most of half an SM's."""
    for vocab in (294920, 300000, 1 << 20):
        p = plan(rows, vocab, k, False, True, True)
        assert p["mode"] == STREAM and sound(p, vocab, k, False, True, True), p


def test_chunks_are_those_of_the_kernel_that_runs(plan):
    """Whole chunks are what the passes take unrolled: as many vectors to a
    thread as the launched kernel is made for.  An SM to itself is a kernel of
    its own only where loss and gradient come from one call; otherwise such a
    CTA runs the half SM's."""
    seen = set()
    for vocab in (4096, 8192, 20000, 50257, 128256, 300000, 1 << 20):
        for k in (0, 64, 500, 555, 600, 767, 900, 1024):
            for f32 in (False, True):
                for grad, first in WAYS:
                    for rows in (1, 40, 8192):
                        p = plan(rows, vocab, k, f32, grad, first)
                        own = p["shape"] == WHOLE and p["mode"] == TRAIN
                        whole = p["threads"] * (3 if own else 2 if f32 else 4)
                        share = -(-(vocab * (4 if f32 else 2) // 16) // p["ctas"])
                        assert p["chunk"] == min(share, whole), (rows, vocab, k, f32, p)
                        seen.add((p["mode"], p["shape"]))
    assert {(m, WHOLE) for m in (FORWARD, TRAIN, STREAM)} <= seen
