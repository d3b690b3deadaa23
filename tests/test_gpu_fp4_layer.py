"""moe_layer_forward_fp4 through its wrapper: buffers larger than the call, tensors that the
wrappers make for a call on another stream."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, NV = 0, 1
BLOCK = {0: 32, 1: 16}


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def scale1(v):
    return torch.full((1,), float(v), device=DEV)


def operand(rng, shape, K, fmt):
    codes = rng.integers(0, 256, (*shape, K // 2), dtype=np.uint8)
    if fmt == MX:
        scales = rng.integers(119, 124, (*shape, K // 32)).astype(np.uint8)
    else:
        scales = rng.integers(0, 0x50, (*shape, K // 16)).astype(np.uint8)
    return dev(codes), dev(scales)


def experts(rng, E, H, I, fmt):
    one = torch.full((E,), 0.05, device=DEV)
    return (*operand(rng, (E, 2 * I), H, fmt), one), (*operand(rng, (E, H), I, fmt), one)


def tokens(rng, T, k, E, H):
    x = dev(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    ids = dev(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32))
    return x, ids, dev(rng.random((T, k)).astype(np.float32))


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
def test_larger_buffers_give_the_same_bits(B, fmt):
    rng = np.random.default_rng(fmt)
    E, H, I = 5, 288, 96
    w13, w2 = experts(rng, E, H, I, fmt)
    kw = dict(x_scale_2=scale1(0.004), h_scale_2=scale1(0.01))
    big = B.LayerBuffersFp4(70, 3, E, H, I, fmt, DEV)
    for T, k in ((70, 3), (1, 1), (70, 2), (33, 3), (64, 3)):
        args = (*tokens(rng, T, k, E, H), w13, w2)
        want = B.layer_forward_fp4(*args, B.LayerBuffersFp4(T, k, E, H, I, fmt, DEV), **kw)
        big.out.fill_(7.0)
        big.y2.fill_(7.0)
        got = B.layer_forward_fp4(*args, big, **kw)
        assert B.read_status(big.workspace) == B.MOE_OK
        assert torch.equal(got, want)
        assert bool((big.out[T:] == 7.0).all()) and bool((big.y2[T * k:] == 7.0).all())


def test_a_call_on_another_stream_leaves_later_memory_alone(B):
    """The side stream is held up, so a workspace made for the call is cleared late: memory
    that the current stream takes meanwhile keeps its contents."""
    rng = np.random.default_rng(2)
    codes, scales = operand(rng, (9,), 64, MX)
    w, wsc = operand(rng, (2, 40), 64, MX)
    sizes = dev(np.array([9, 0], np.int32))
    want = B.fp4_grouped_gemm(codes, scales, w, wsc, sizes, MX)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = B.fp4_grouped_gemm(codes, scales, w, wsc, sizes, MX, stream=side)
    later = [torch.full((256,), 7, dtype=torch.uint8, device=DEV) for _ in range(64)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((t == 7).all()) for t in later)


def test_a_stream_given_by_its_handle(B):
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    x = torch.randn((5, 64), device=DEV)
    want = B.fp4_quantize(x, MX)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = B.fp4_quantize(x, MX, stream=Handle(side))
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
