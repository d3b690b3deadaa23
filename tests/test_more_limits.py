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


CAPACITY = 6
MOST = 2 ** 19


def test_sums_too_long_for_the_tensor_cores_f32_are_refused(lib):
    """A tensor core cuts off what a sum's f32 does not hold, up to a step in eight products: K 2^-27
    of the sum where all have one sign (5% were gone at K = 2^23), and an item of some 4e8 tokens
    outlasts a wait's 2 s.  K up to 2^19 stays within half a step of bf16."""
    stop = (UNSUPPORTED, CUDA)

    def forward(T=5, hidden=64, inter=32, w13=FAKE):
        return lib.moe_ffn_forward(FAKE, hidden, T, hidden, inter, w13, FAKE, FAKE, FAKE, FAKE, 1, FAKE, 256, None)

    def backward(T=5, hidden=64, inter=32, dx=FAKE, dw13=FAKE, dw2=FAKE, dout=FAKE):
        return lib.moe_ffn_backward(dout, FAKE, hidden, T, hidden, inter, FAKE, FAKE, FAKE, FAKE, FAKE, dx, dw13, dw2, 1, FAKE,
                                    256, None)

    for f in (forward, backward):
        assert f(hidden=MOST + 8) == CAPACITY and f(inter=MOST // 2 + 8) == CAPACITY
    assert backward(T=MOST + 1) == CAPACITY
    assert backward(T=MOST + 1, dw13=None) == CAPACITY and backward(T=MOST + 1, dw2=None) == CAPACITY
    assert backward(T=2 ** 30 - 1, dx=None) == CAPACITY
    # an invalid argument comes first
    assert forward(hidden=MOST + 8, w13=None) == INVALID and backward(T=MOST + 1, dout=None) == INVALID
    if not torch.cuda.is_available():                           # these stop at the device
        assert forward(hidden=MOST, inter=MOST // 2) in stop and forward(T=2 ** 30 - 1) in stop
        assert backward(T=MOST) in stop and backward(T=2 ** 30 - 1, dw13=None, dw2=None) in stop
