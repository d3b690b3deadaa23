"""Few-row MXFP4 products over the whole range of the scale's byte, against 64 bits.

Tolerance: 1e-5 sum|x w| for f32 sums of exact products (K 2^-24 is 3e-5 as a bound for K = 512, a
sum of rounded steps in practice sqrt(K) 2^-24 = 1.3e-6); elements of x below 2^-28 of their row's
largest are rounded to 2^-38 of it, 2^-39 max|x| sum|w|; and sums lie on f32's grid below 2^-126,
half a step of 2^-149 for each addition over blocks, lanes and warps: 2^-147 a block.  Magnitudes
past f32's are left out."""
import pytest
import torch

pytestmark = pytest.mark.gpu
MAGS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


def dense(codes, scales):
    b = codes.long()
    table = torch.tensor(MAGS + [-m for m in MAGS], dtype=torch.float64, device="cuda")
    v = torch.stack([table[b & 15], table[b >> 4]], dim=-1).flatten(-2)
    powers = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")
    return v * powers[scales.long()].repeat_interleave(32, -1)


# rows of x that an expert has (one or two, up to four, and more go different ways), and whether
# there are other experts
ROWS = [(1, 9), (2, 9), (3, 9), (4, 9), (7, 9), (1, 1), (5, 1), (8, 1)]


@pytest.mark.parametrize("power", [-120, -60, -28, -17, -8, 0, 16, 17, 60, 120])
@pytest.mark.parametrize("rows,E", ROWS)
def test_every_scale_byte(B, rows, E, power):
    """A column a byte, 0 to 252, all of its blocks alike; x at many magnitudes, K off a stage."""
    K, N = 544, 253
    g = torch.Generator(device="cuda").manual_seed(rows * 1000 + E)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.arange(N, device="cuda").to(torch.uint8).view(1, N, 1).repeat(E, 1, K // 32)
    x = (torch.randn((rows, K), generator=g, device="cuda").double() * 2.0 ** power).bfloat16()
    e = E // 2
    ids = torch.full((rows,), e, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = B.fp4_matvec(x, codes, scales, 0, row_expert=ids, workspace=ws).double()
    assert B.read_status(ws) == B.MOE_OK
    W = dense(codes[e], scales[e])
    want, mass = x.double() @ W.T, x.double().abs() @ W.abs().T
    tol = 1e-5 * mass + 2.0 ** -39 * x.double().abs().amax(1, keepdim=True) * W.abs().sum(1) + 2.0 ** -147 * (K // 32)
    fits = mass < 2.0 ** 127
    bad = ((got - want).abs() > tol) & fits
    assert not bool(bad.any()), (bad.nonzero()[:5].tolist(), int(bad.sum()))
    assert int(fits.any(0).sum()) > 100


@pytest.mark.parametrize("rows,E", ROWS)
def test_blocks_of_far_apart_scales(B, rows, E):
    """Bytes of one column from both ends, rows of x of different magnitudes in one call."""
    K, N = 1024, 40
    g = torch.Generator(device="cuda").manual_seed(rows + E)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0, 253, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    scales[:, :20] //= 12                                         # 0 to 21: all small
    x = torch.randn((rows, K), generator=g, device="cuda").double()
    x *= 2.0 ** torch.tensor([0, -20, 30, 9, -100, -4, 60, 2], dtype=torch.float64, device="cuda")[:rows, None]
    x = x.bfloat16()
    e = E // 2
    ids = torch.full((rows,), e, dtype=torch.int32, device="cuda")
    got = B.fp4_matvec(x, codes, scales, 0, row_expert=ids).double()
    W = dense(codes[e], scales[e])
    want, mass = x.double() @ W.T, x.double().abs() @ W.abs().T
    tol = 1e-5 * mass + 2.0 ** -39 * x.double().abs().amax(1, keepdim=True) * W.abs().sum(1) + 2.0 ** -147 * (K // 32)
    assert bool((((got - want).abs() <= tol) | (mass >= 2.0 ** 127)).all())


@pytest.mark.parametrize("rows", [1, 3])
def test_a_zero_block_of_the_largest_scale_beside_large_x(B, rows):
    """0 times a scale that x's magnitude would carry past f32 is 0."""
    K = 64
    codes = torch.zeros((2, 8, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((2, 8, 2), 252, dtype=torch.uint8, device="cuda")
    scales[..., 1] = 100
    codes[..., 20] = 0x22                                         # two ones in the second block
    x = torch.full((rows, K), 2.0 ** 100, device="cuda").bfloat16()
    ids = torch.ones(rows, dtype=torch.int32, device="cuda")
    got = B.fp4_matvec(x, codes, scales, 0, row_expert=ids)
    assert bool((got == 2.0 ** 101 * 2.0 ** -27).all())
