"""Gradients of weights over as many tokens as the dense block takes, against sums in 64 bits.

Tolerance: a tensor core cuts off what the f32 of a sum does not hold, up to a step (2^-23) in
eight products, of what has been summed by then: where all have one sign K / 16 2^-23 = K 2^-27 of
the sum, otherwise at most that of the sum of magnitudes.  2^-8 for K = 2^19."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("T", [2 ** 14 + 3, 2 ** 19])
@pytest.mark.parametrize("one_sign", [False, True])
def test_weight_gradients_of_many_tokens(B, T, one_sign):
    g = torch.Generator(device="cuda").manual_seed(T)
    H, I = 24, 16

    def make(*shape):
        t = torch.randn(shape, generator=g, device="cuda").bfloat16()
        return t.abs() if one_sign else t

    dout, x, h = make(T, H), make(T, H), make(T, I)
    w13, w2, gu = make(2 * I, H), make(H, I), make(T, 2 * I)
    dgu = torch.empty_like(gu)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dx, dw13, dw2 = B.ffn_backward(dout, x, w13, w2, h, gu, dgu=dgu, dw_dtype=torch.float32, workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    for got, a, b in ((dw2, dout, h), (dw13, dgu, x)):
        a, b = a.double(), b.double()
        assert bool(((got.double() - a.T @ b).abs() <= T * 2.0 ** -27 * (a.abs().T @ b.abs())).all())


def test_more_tokens_are_refused(B):
    T, H, I = 2 ** 19 + 1, 8, 8
    x, w13, w2 = (torch.zeros(s, device="cuda").bfloat16() for s in ((T, H), (2 * I, H), (H, I)))
    gu = torch.zeros((T, 2 * I), device="cuda").bfloat16()
    with pytest.raises(B.MoeError) as e:
        B.ffn_backward(x, x, w13, w2, x, gu)
    assert e.value.status == 6
    dx, a, b = B.ffn_backward(x, x, w13, w2, x, gu, out=(torch.ones_like(x), None, None))     # dx alone sums over 2 I
    assert a is None and b is None and bool((dx == 0).all())
