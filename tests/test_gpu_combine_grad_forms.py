"""moe_combine_backward with one of its two outputs left out (NULL): the same bits as together,
and y may be NULL where no weight gradient is asked for."""
import numpy as np
import pytest
import torch

from fp4_weight_grouped_gb300 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


def call(B, dout, y, s2r, w, N, dy, dw):
    code = lambda t: B.MOE_F32 if t is None or t.dtype == F32 else B.MOE_BF16  # noqa: E731
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    T, k = w.shape
    return B.load().moe_combine_backward(ptr(dout), code(dout), ptr(y), code(y), ptr(s2r), ptr(w), T, k, N, ptr(dy),
                                         code(dy), ptr(dw), torch.cuda.current_stream().cuda_stream)


# A warp a slot, fewer lanes, a block a slot; vectors of 8, 4 and 1.
@pytest.mark.parametrize("T,E,k,N", [(130, 8, 8, 4096), (1200, 16, 2, 260), (200, 8, 3, 72), (9, 8, 4, 12), (33, 8, 2, 3),
                                     (3, 4, 2, 1024), (64, 8, 6, 516), (5, 8, 2, 131)])
@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, F32, BF16), (BF16, BF16, BF16)],
                         ids=lambda t: "-".join(str(x)[6:] for x in t))
def test_each_gradient_alone(B, T, E, k, N, types):
    gen = torch.Generator(device=DEV).manual_seed(T + N)
    ids = inputs.route_uniform(T, T, E, k)
    ids.reshape(-1)[1::7] = -1                           # slots without a row
    s2r = B.route_sort(torch.from_numpy(np.ascontiguousarray(ids)).to(DEV), E)[3]
    w = torch.rand((T, k), generator=gen, device=DEV)
    dout = torch.randn((T, N), generator=gen, device=DEV).to(types[0])
    y = torch.randn((T * k, N), generator=gen, device=DEV).to(types[1])

    def outputs():
        return torch.full((T * k, N), 7.0, dtype=types[2], device=DEV), torch.full((T, k), 7.0, device=DEV)

    both, dy, dw = outputs(), outputs()[0], outputs()[1]
    assert call(B, dout, y, s2r, w, N, *both) == B.MOE_OK
    assert call(B, dout, None, s2r, w, N, dy, None) == B.MOE_OK
    assert call(B, dout, y, s2r, w, N, None, dw) == B.MOE_OK
    assert torch.equal(dy, both[0]) and torch.equal(dw, both[1])
