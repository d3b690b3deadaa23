"""Sizes at the ends of what the few-row products, the dense block and the clipping take,
without a GPU: only calls that are rejected before any device work are made (the pointers are
not device memory), and rules that the kernels share are compiled from their own headers."""
import pytest
import torch

from fp4_weight_grouped_gb300 import binding, build_lib

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
