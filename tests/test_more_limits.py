"""Sizes at the ends of what the few-row products, the dense block and the clipping take,
without a GPU: only calls that are rejected before any device work are made (the pointers are
not device memory), and rules that the kernels share are compiled from their own headers."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from fp4_weight_grouped_gb300 import binding, build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, CUDA = 1, 2, 3
FAKE = 4096


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


def matvec(lib, N, rows=1, E=1):
    return lib.moe_fp4_matvec(FAKE, 32, 1, None, rows, 32, FAKE, FAKE, None, 0, E, N, FAKE, 0, FAKE, 256, None)


def test_columns_that_a_tile_s_numbers_cannot_hold_are_refused(lib):
    """A tile's last column, and those of the tiles behind it in its item, are 32-bit numbers: up to
    510 past N.  With more columns the tiles' count came out negative and no output was written."""
    assert all(matvec(lib, N) == INVALID for N in (2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 512))
    if not torch.cuda.is_available():                          # the others stop at the device
        assert matvec(lib, 2 ** 31 - 513) in (UNSUPPORTED, CUDA)
        # half as many columns of h: nothing there is near the limit
        assert lib.moe_fp4_matvec_swiglu(FAKE, 32, 1, None, 1, 32, FAKE, FAKE, None, 0, 1, 2 ** 30 - 1, FAKE, FAKE, 256,
                                         None) in (UNSUPPORTED, CUDA)


@pytest.fixture(scope="module")
def accumulator_limit(tmp_path_factory):
    d = tmp_path_factory.mktemp("limit")
    src, so = d / "limit.cpp", d / "limit.so"
    src.write_text('#include "pair_schedule.h"\nextern "C" uint64_t limit(uint64_t ns, int k_stages) '
                   "{ return moe::accumulator_limit(ns, k_stages); }\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{ROOT}/fp4_weight_grouped_gb300/csrc", str(src), "-o",
                    str(so)], check=True)
    f = C.CDLL(str(so)).limit
    f.argtypes, f.restype = [C.c_uint64, C.c_int], C.c_uint64
    return f


def test_the_wait_for_an_accumulator_grows_with_its_k(accumulator_limit):
    """An epilogue waits for all of an item's K, which for the gradients of weights is the tokens: up
    to 2^30.  A stage of 64 k takes up to 0.33 us; by a limit of 2 s alone, whatever K, a backward of
    some 4e8 tokens gave up in the middle of its work.  Five times the stages' time beside the 2 s."""
    s = 2_000_000_000
    for tokens in (1, 8192, 2 ** 26, 6 * 10 ** 8, 2 ** 30 - 1):
        stages = -(-tokens // 64)
        assert s + 5 * 330 * stages <= accumulator_limit(s, stages) <= s + 10_000 * stages
