"""q8_prepare_device() when a part of the set-up fails: the library's own host
code, linked with set-up functions that fail on demand.  No GPU is needed."""
import ctypes as C
import glob
import os
import subprocess

import pytest

from bit_blockwise_adamw_gb300 import build

STEPS = ["device_tables", "prepare_step8", "prepare_step1", "prepare_step16", "prepare_codec"]
OPERATORS = ["prepare_ff", "prepare_norm", "prepare_distill"]

FAKES = r"""
#include "q8_internal.h"
#include "q8_train.h"
static int g_failing = -1, g_calls = 0;
extern "C" int fake_failing(int which) { const int n = g_calls; g_failing = which; g_calls = 0; return n; }
namespace q8 {
static cudaError_t part(int which) { ++g_calls; return which == g_failing ? cudaErrorNotSupported : cudaSuccess; }
cudaError_t device_tables(const DevTables** out) { *out = nullptr; return part(0); }
cudaError_t prepare_step8() { return part(1); }
cudaError_t prepare_step1() { return part(2); }
cudaError_t prepare_step16() { return part(3); }
cudaError_t prepare_codec() { return part(4); }
cudaError_t prepare_ff() { return part(5); }
cudaError_t prepare_norm() { return part(6); }
cudaError_t prepare_distill() { return part(7); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    objects = sorted(glob.glob(os.path.join(build.OUT_DIR, "*.cu.o")))
    d = tmp_path_factory.mktemp("fakes")
    src, so = str(d / "fakes.cu"), str(d / "libfakes.so")
    with open(src, "w") as f:
        f.write(FAKES)
    # the fakes stand before the library's own definitions
    subprocess.run([build.nvcc(), *build.NVCC_FLAGS, "-shared", src, *objects, "-Xlinker", "--allow-multiple-definition", "-o", so],
                   check=True)
    lib = C.CDLL(so)
    lib.q8_last_error.restype = C.c_char_p
    return lib


@pytest.mark.parametrize("part", OPERATORS)
def test_a_step_does_not_need_the_training_step_operators(lib, part):
    """The optimizers' set-up stands where that of an operator around them
    cannot be had; all other parts are still set up."""
    lib.fake_failing((STEPS + OPERATORS).index(part))
    assert lib.q8_prepare_device() == 0
    assert lib.fake_failing(-1) == len(STEPS + OPERATORS)


@pytest.mark.parametrize("part", STEPS)
def test_a_failing_step_is_reported(lib, part):
    lib.fake_failing(STEPS.index(part))
    assert lib.q8_prepare_device() == -5
    assert b"q8_prepare_device" in lib.q8_last_error()
    lib.fake_failing(-1)
    assert lib.q8_prepare_device() == 0
