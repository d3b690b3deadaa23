"""4-bit activations: moe_fp4_quantize and the W4A4 grouped products against plain
64-bit implementations written here from the formats' definitions.

Tolerances, fixed before the first run:
  quantiser   MXFP4 bit-exact (its scaling is a power of two, so only the nearest-code
              step rounds); NVFP4 bit-exact against its stated float32 steps, each of
              which is one IEEE operation.
  products    |gpu - exact| <= 1e-5 * sum_k |a w| + 1e-6, the library's bound for f32
              sums (bf16 outputs: one bf16 ulp more).
  SwiGLU      with u the block's step 2^(byte - 127) (or s g), d(m) the distance from m
              to the nearest e2m1 magnitude and tau the f32 error of h before rounding:
              |h_q - h| <= u d(|h| / u) + 2 tau (the nearest code to h + e, |e| <= tau,
              is at most d(h) + |e| away from h + e); the scale byte is one that some
              h within tau gives.
"""
import numpy as np
import pytest
import torch

from parity_bounds import SILU_SLOPE_MAX, bf16_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"
MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([MAGS, -MAGS])
BLOCK = {0: 32, 1: 16}
MX, NV = 0, 1


@pytest.fixture(params=["auto", "on"])
def pairing(B, request):
    """Small calls run long bands in one launch with the short ones; "on" splits them as
    large calls do."""
    B.set_gemm_pairing(B.MOE_PAIRING_ON if request.param == "on" else B.MOE_PAIRING_AUTO)
    yield
    B.set_gemm_pairing(B.MOE_PAIRING_AUTO)


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


# ------------------------------------------------------- plain definitions

def e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_values()


def scale_values(bytes_, fmt):
    return np.ldexp(1.0, bytes_.astype(np.int64) - 127) if fmt == MX else E4M3[bytes_]


def values(codes, scales, fmt):
    """Codes uint8 [..., K/2] and block scales -> float64 [..., K]."""
    nib = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    return E2M1[nib] * np.repeat(scale_values(scales, fmt), BLOCK[fmt], axis=-1)


def nearest_code(q):
    """e2m1 code nearest to q (float64 exact of a float32), ties to the even mantissa."""
    m = np.abs(q)
    c = ((m > 0.25).astype(np.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5)
         + (m > 5.0)).astype(np.uint8)
    return np.where((q < 0) & (c > 0), c | 8, c)


def nearest_e4m3(t):
    """Non-negative float32 <= 448 -> E4M3 byte, nearest, ties to even."""
    t = t.astype(np.float64)
    pos = E4M3[:127]
    hi = np.clip(np.searchsorted(pos, t), 1, 126)
    lo = hi - 1
    dl, dh = t - pos[lo], pos[hi] - t
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi))).astype(np.uint8)


def quantise(x, fmt, g=np.float32(1)):
    """float32 [rows, K] -> codes, scale bytes (finite input, or NaN-marked blocks)."""
    rows, K = x.shape
    xb = x.reshape(rows, K // BLOCK[fmt], BLOCK[fmt])
    bad = ~np.isfinite(xb).all(-1)
    xb = np.where(bad[..., None], np.float32(0), xb)
    a = np.abs(xb).max(-1)
    if fmt == MX:
        _, e = np.frexp(a.astype(np.float64))
        byte = np.where(a == 0, 0, np.clip(e - 1 - 2 + 127, 0, 252))
        q = np.ldexp(xb.astype(np.float64), (127 - byte)[..., None])
        nan = 255
    else:
        g = np.float32(g)
        byte = nearest_e4m3(np.minimum(a / (np.float32(6) * g), np.float32(448)))
        with np.errstate(divide="ignore", over="ignore"):
            r = np.float32(1) / (E4M3[byte].astype(np.float32) * g)
        r = np.where(np.isfinite(r), r, np.float32(0))
        q = (xb * r[..., None]).astype(np.float32).astype(np.float64)
        nan = 127
    codes = nearest_code(q)
    codes = np.where(bad[..., None], 0, codes).reshape(rows, K)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), np.where(bad, nan, byte).astype(np.uint8)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def scale1(v):
    return torch.full((1,), float(v), device=DEV)


def status_ws():
    return torch.zeros(256, dtype=torch.uint8, device=DEV)


# -------------------------------------------------------------- quantiser

def awkward_rows(rng, rows, K):
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x *= np.exp2(rng.integers(-30, 30, (rows, K // 16))).astype(np.float32).repeat(16, 1)
    flat = x.reshape(-1, 16)
    n = flat.shape[0]
    flat[0] = 0                                               # all zeros
    flat[1 % n] = np.tile(np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]), 2)   # ties
    flat[2 % n] = -flat[1 % n]
    flat[3 % n, ::2] = -0.0
    return x


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (7, 288), (130, 1056), (33, 4096)])
def test_quantize_bit_exact(B, fmt, bf16, rows, K):
    rng = np.random.default_rng(rows * K + fmt)
    x = awkward_rows(rng, rows, K)
    t = dev(x)
    if bf16:
        t = t.to(torch.bfloat16)
        x = t.float().cpu().numpy()
    g = np.float32(0.37)
    ws = status_ws()
    vals = torch.empty((rows, K), device=DEV)
    codes, scales = B.fp4_quantize(t, fmt, tensor_scale=scale1(g), values=vals, workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    rc, rs = quantise(x, fmt, g)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    v = values(rc, rs, fmt)
    if fmt == NV:
        v = (v.astype(np.float32) * g).astype(np.float32)     # one rounding, by g
    np.testing.assert_array_equal(vals.cpu().numpy().astype(np.float64), v.astype(np.float64))


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
def test_quantize_gather_strides_and_alignment(B, fmt):
    """Row index with a divisor, a padded row stride, and a base off 16 bytes give what
    the contiguous rows give."""
    rng = np.random.default_rng(5)
    T, k, K = 41, 3, 96
    x = dev(awkward_rows(rng, T, K)).to(torch.bfloat16)
    order = dev(rng.permutation(T * k).astype(np.int32))
    g = scale1(0.01)
    want = B.fp4_quantize(x[(order // k).long()].contiguous(), fmt, tensor_scale=g)
    for off, pad in ((0, 0), (0, 8), (1, 3), (5, 11)):
        big = torch.zeros((T, K + pad + off), dtype=torch.bfloat16, device=DEV)
        big[:, off:off + K] = x
        view = big[:, off:off + K]
        got = B.fp4_quantize(view, fmt, row_index=order, index_div=k, tensor_scale=g)
        for a, b in zip(got, want):
            assert torch.equal(a, b), (off, pad)


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_quantize_many_rows_repeat_few(B, fmt, dtype):
    """More rows than the GPU holds warps for, gathered from 130, some without a source, with
    x and values 32-byte, 16-byte and element aligned: each row is its source's, bit for bit."""
    rng = np.random.default_rng(11 + fmt)
    T, rows, K = 130, 40001, 1056
    x = dev(awkward_rows(rng, T, K)).to(dtype)
    g = scale1(0.37)
    one = torch.empty((T, K), dtype=dtype, device=DEV)
    wc, wsc = B.fp4_quantize(x, fmt, tensor_scale=g, values=one)
    pick = rng.integers(0, T, rows).astype(np.int32)
    pick[::997] = T                                  # past the last row
    at, there = dev(pick), dev(pick < T)
    src = at.long().clamp_max(T - 1)
    piece = 16 // x.element_size()
    for off in (0, piece, 1):
        big = torch.zeros((T, K + 2 * piece), dtype=dtype, device=DEV)
        view = big[:, off:off + K]
        view.copy_(x)
        buf = torch.zeros(rows * K + 2 * piece, dtype=dtype, device=DEV)
        v = buf[off if off != 1 else 0:][:rows * K].view(rows, K)
        ws = status_ws()
        c, sc = B.fp4_quantize(view, fmt, row_index=at, tensor_scale=g, values=v, workspace=ws)
        assert B.read_status(ws) == B.MOE_ERR_DATA
        assert torch.equal(c, wc[src] * there[:, None]) and torch.equal(sc, wsc[src] * there[:, None])
        assert torch.equal(v[there], one[src][there]) and int(torch.count_nonzero(v[~there])) == 0
        c, sc = B.fp4_quantize(view, fmt, row_index=at, tensor_scale=g)
        assert torch.equal(c, wc[src] * there[:, None]) and torch.equal(sc, wsc[src] * there[:, None])


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
def test_quantize_extremes_and_nonfinite(B, fmt):
    x = np.zeros((9, 64), np.float32)
    x[0] = np.finfo(np.float32).max
    x[1] = np.float32(2.0) ** -149                   # smallest subnormal
    x[2] = np.float32(2.0) ** -126
    x[3, 5] = np.inf
    x[4, 40] = -np.inf
    x[5, 0] = np.nan
    x[6, ::7] = -0.0
    x[7, 33] = 1e-30
    x[8] = np.linspace(-7, 7, 64)
    ws = status_ws()
    g = np.float32(0.5)
    codes, scales = B.fp4_quantize(dev(x), fmt, tensor_scale=scale1(g), workspace=ws)
    rc, rs = quantise(x, fmt, g)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    assert B.read_status(ws) == B.MOE_OK


def test_quantize_index_out_of_range_and_bad_scale(B):
    x = torch.randn((4, 64), device=DEV)
    for bad in (-1, 8, 2 ** 31 - 1):
        ws = status_ws()
        idx = dev(np.array([0, bad, 3], np.int32))
        codes, scales = B.fp4_quantize(x, MX, row_index=idx, index_div=2, workspace=ws)
        assert B.read_status(ws) == B.MOE_ERR_DATA
        want = B.fp4_quantize(x[[0, 1]].contiguous(), MX)
        assert torch.equal(codes[[0, 2]], want[0]) and torch.equal(scales[[0, 2]], want[1])
        assert int(codes[1].max()) == 0 and int(scales[1].max()) == 0
    for g in (0.0, -1.0, float("inf"), float("nan")):
        ws = status_ws()
        B.fp4_quantize(x, NV, tensor_scale=scale1(g), workspace=ws)
        assert B.read_status(ws) == B.MOE_ERR_DATA


# ---------------------------------------------------------------- products

def random_operand(rng, shape, K, fmt, lo=-8, hi=-4):
    codes = rng.integers(0, 256, (*shape, K // 2), dtype=np.uint8)
    if fmt == MX:
        scales = (127 + rng.integers(lo, hi + 1, (*shape, K // 32))).astype(np.uint8)
    else:
        scales = rng.integers(0, 0x50, (*shape, K // 16)).astype(np.uint8)
    return codes, scales


def check_product(B, rng, fmt, sizes, K, N, out_dtype=torch.float32, wide=False, offset=0, stream=None):
    E, rows = len(sizes), int(np.sum(sizes))
    span = dict(lo=-40, hi=40) if wide else {}
    ac, asc = random_operand(rng, (rows,), K, fmt, **span)
    wc, wsc = random_operand(rng, (E, N), K, fmt, **span)
    a2, w2 = np.float32(0.75), (rng.random(E) + 0.5).astype(np.float32)

    def scales_at(s):      # scale bytes at an address `offset` past an aligned one
        buf = torch.zeros(s.size + 64, dtype=torch.uint8, device=DEV)
        v = buf[offset:offset + s.size].view(s.shape)
        v.copy_(dev(s))
        return v

    ws = status_ws()
    args = (dev(ac), scales_at(asc), dev(wc), scales_at(wsc), dev(np.asarray(sizes, np.int32)), fmt)
    out = torch.full((rows, N), 7.0, dtype=out_dtype, device=DEV)
    torch.cuda.synchronize()
    B.fp4_grouped_gemm(*args, act_scale_2=scale1(a2), weight_scale_2=dev(w2), out=out, workspace=ws, stream=stream)
    assert B.read_status(ws, stream) == B.MOE_OK
    a = values(ac, asc, fmt)
    r = 0
    got = out.double().cpu().numpy()
    for e, n in enumerate(sizes):
        if n == 0:
            continue
        w = values(wc[e], wsc[e], fmt)
        s = float(a2 * w2[e]) if fmt == NV else 1.0
        ref, mag = a[r:r + n] @ w.T * s, np.abs(a[r:r + n]) @ np.abs(w).T * s
        bound = 1e-5 * mag + 1e-6
        if out_dtype == torch.bfloat16:
            bound = bound + bf16_ulp(ref)
        diff = np.abs(got[r:r + n] - ref)
        assert np.all(diff <= bound), (e, n, float((diff / bound).max()))
        r += n
    return args, out


SIZES = [
    ([1], 32, 1), ([5], 64, 130), ([0, 3, 0], 96, 128), ([17, 1, 0, 40], 256, 129),
    ([16, 33, 65], 512, 384), ([129, 0, 193, 385], 288, 200), ([192, 191, 1], 1056, 260),
    ([200, 3, 0, 193, 192, 1, 600, 512], 288, 200), ([700, 1, 900, 16], 1056, 456), ([257, 1300, 0, 40], 2048, 192),
    ([193], 96, 40), ([700], 768, 136), ([192, 400], 4096, 128), ([2] * 40 + [0] * 5 + [90], 512, 256), ([1], 8192, 256),
]


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("sizes,K,N", SIZES, ids=[f"E{len(s)}_K{k}_N{n}" for s, k, n in SIZES])
def test_product_matches_64_bits(B, pairing, fmt, sizes, K, N):
    rng = np.random.default_rng(K + N + fmt)
    check_product(B, rng, fmt, sizes, K, N)
    check_product(B, rng, fmt, sizes, K, N, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_product_scale_alignment(B, pairing, fmt, offset):
    check_product(B, np.random.default_rng(offset), fmt, [30, 0, 70], 512, 140, offset=offset)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [203, 204, 216])
def test_product_output_alignment_of_long_bands(B, pairing, N, dtype):
    """Rows and bases of every alignment give the same sums, and nothing outside the
    output is written."""
    rng = np.random.default_rng(N)
    args, out = check_product(B, rng, MX, [300, 0, 40, 1000], 96, N, out_dtype=dtype)
    for off in (1, 4, 8, 16):
        flat = torch.full((out.numel() + 64,), 7.0, dtype=dtype, device=DEV)
        got = flat[off:off + out.numel()].view(out.shape)
        B.fp4_grouped_gemm(*args, out=got)
        assert torch.equal(got, out)
        assert bool((flat[:off] == 7.0).all()) and bool((flat[off + out.numel():] == 7.0).all())


def test_product_wide_scale_range(B):
    check_product(B, np.random.default_rng(3), MX, [9, 50], 256, 128, wide=True)


def test_product_many_experts_and_side_stream(B):
    rng = np.random.default_rng(4)
    sizes = rng.integers(0, 4, 1024).tolist()
    check_product(B, rng, MX, sizes, 64, 8)
    s = torch.cuda.Stream()
    check_product(B, rng, NV, [3, 0, 21], 320, 72, stream=s)


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
def test_product_repeats_bit_for_bit(B, pairing, fmt):
    rng = np.random.default_rng(8)
    args, out = check_product(B, rng, fmt, rng.integers(0, 300, 24).tolist(), 1024, 384)
    a2, w2 = scale1(0.75), None
    if fmt == NV:
        w2 = torch.ones(24, device=DEV)
    first = B.fp4_grouped_gemm(*args, act_scale_2=a2, weight_scale_2=w2)
    for _ in range(20):
        assert torch.equal(first, B.fp4_grouped_gemm(*args, act_scale_2=a2, weight_scale_2=w2))


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
def test_long_bands_repeat_bit_for_bit(B, pairing, fmt):
    """Bands of every length class, forty times: a race in a ring shows as a difference."""
    rng = np.random.default_rng(18)
    sizes = rng.integers(0, 700, 12).tolist()
    args, _ = check_product(B, rng, fmt, sizes, 1536, 448)
    kw = dict(act_scale_2=scale1(0.75), weight_scale_2=torch.ones(12, device=DEV))
    first = B.fp4_grouped_gemm(*args, **kw)
    gated = B.fp4_grouped_gemm_swiglu(*args, h_scale_2=scale1(0.02), **kw)
    for _ in range(40):
        assert torch.equal(first, B.fp4_grouped_gemm(*args, **kw))
        for a, b in zip(gated, B.fp4_grouped_gemm_swiglu(*args, h_scale_2=scale1(0.02), **kw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("K", [96, 1056, 2048])
def test_cta_pairs_and_graphs_give_the_same_bits(B, pairing, fmt, K):
    """Bands of every length in CTA pairs or not, and replayed from a CUDA graph (whose
    reader must wait for both launches), on outputs that are cleared before each replay."""
    rng = np.random.default_rng(K)
    sizes = [700, 3, 0, 161, 250, 31, 112, 1000]
    E, N, rows = len(sizes), 448, sum(sizes)
    ac, asc = random_operand(rng, (rows,), K, fmt)
    wc, wsc = random_operand(rng, (E, N), K, fmt)
    args = (dev(ac), dev(asc), dev(wc), dev(wsc), dev(np.array(sizes, np.int32)), fmt)
    kw = dict(act_scale_2=scale1(0.5), weight_scale_2=torch.ones(E, device=DEV), workspace=status_ws())
    h2 = scale1(0.02)
    out = torch.empty((rows, N), device=DEV)
    h = (torch.empty((rows, N // 4), dtype=torch.uint8, device=DEV),
         torch.empty((rows, N // 2 // BLOCK[fmt]), dtype=torch.uint8, device=DEV))
    sums = torch.empty((), dtype=torch.float64, device=DEV)

    def run():
        out.zero_()
        B.fp4_grouped_gemm(*args, out=out, **kw)
        sums.copy_(out.double().sum())
        h[0].zero_()
        B.fp4_grouped_gemm_swiglu(*args, h_scale_2=h2, out=h, **kw)

    run()
    want = [t.clone() for t in (out, sums, *h)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, sums, *h)))
    B.set_gemm_pairing(B.MOE_PAIRING_OFF)
    run()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, sums, *h)))


def test_product_no_rows_and_bad_sizes(B):
    rng = np.random.default_rng(9)
    wc, wsc = random_operand(rng, (3, 64), 64, MX)
    ac, asc = random_operand(rng, (10,), 64, MX)
    ws = status_ws()
    z = B.fp4_grouped_gemm(dev(ac[:0]), dev(asc[:0]), dev(wc), dev(wsc), dev(np.zeros(3, np.int32)), MX,
                           workspace=ws)
    assert z.shape == (0, 64) and B.read_status(ws) == B.MOE_OK
    for sizes in ([5, 4, 0], [5, 4, 2], [11, -1, 0], [2 ** 31 - 1, 2 ** 31 - 1, 12]):
        ws = status_ws()
        out = torch.full((10, 64), 3.0, device=DEV)
        B.fp4_grouped_gemm(dev(ac), dev(asc), dev(wc), dev(wsc), dev(np.array(sizes, np.int32)), MX, out=out,
                           workspace=ws)
        assert B.read_status(ws) == B.MOE_ERR_DATA
        assert bool((out == 3.0).all())


@pytest.mark.parametrize("fmt,byte", [(MX, 255), (NV, 0x7F), (NV, 0xFF), (NV, 0x9A)])
@pytest.mark.parametrize("side", ["act", "weight"])
def test_product_reports_bad_scales(B, pairing, fmt, byte, side):
    """Only the row (or column) of the bad scale may differ from a clean run."""
    rng = np.random.default_rng(10)
    wc, wsc = random_operand(rng, (2, 70), 160, fmt)
    ac, asc = random_operand(rng, (30,), 160, fmt)
    kw = dict(act_scale_2=scale1(1), weight_scale_2=torch.ones(2, device=DEV))
    gs = dev(np.array([13, 17], np.int32))
    clean = B.fp4_grouped_gemm(dev(ac), dev(asc), dev(wc), dev(wsc), gs, fmt, **kw)
    (asc[20] if side == "act" else wsc[1, 69])[3] = byte
    ws = status_ws()
    out = B.fp4_grouped_gemm(dev(ac), dev(asc), dev(wc), dev(wsc), gs, fmt, workspace=ws, **kw)
    assert B.read_status(ws) == B.MOE_ERR_DATA
    keep = torch.ones((30, 70), dtype=torch.bool, device=DEV)
    if side == "act":
        keep[20] = False
    else:
        keep[13:, 69] = False
    assert torch.equal(out[keep], clean[keep])


def test_product_offsets_past_32_bits(B):
    """rows * N over 2^31 outputs: the last rows against the definition."""
    rng = np.random.default_rng(11)
    rows, N, K = 70016, 32768, 32
    ac, asc = random_operand(rng, (rows,), K, MX)
    wc, wsc = random_operand(rng, (1, N), K, MX)
    ws = status_ws()
    out = B.fp4_grouped_gemm(dev(ac), dev(asc), dev(wc), dev(wsc), dev(np.array([rows], np.int32)), MX,
                             out_dtype=torch.bfloat16, workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    for r in (slice(0, 3), slice(65530, 65540), slice(rows - 5, rows)):
        a, w = values(ac[r], asc[r], MX), values(wc[0], wsc[0], MX)
        ref, mag = a @ w.T, np.abs(a) @ np.abs(w).T
        assert np.all(np.abs(out[r].double().cpu().numpy() - ref) <= 1e-5 * mag + 1e-6 + bf16_ulp(ref))


# ------------------------------------------------- fused SwiGLU and the layer

def nearest_distance(m):
    return np.abs(np.minimum(m, 1e30)[..., None] - MAGS).min(-1)


def swiglu_reference(a, w, I, s):
    y, mag = a @ w.T * s, np.abs(a) @ np.abs(w).T * s
    g, u = y[:, :I], y[:, I:]
    tg, tu = 1e-5 * mag[:, :I] + 1e-6, 1e-5 * mag[:, I:] + 1e-6
    silu = g / (1 + np.exp(-g))
    h = silu * u
    # f32 rounding of silu (a few ulps) and of the product on top of the sums' bounds
    return h, SILU_SLOPE_MAX * tg * (np.abs(u) + tu) + np.abs(silu) * tu + 2.0 ** -20 * np.abs(h)


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("sizes,K,I", [([1], 32, 32), ([5, 0, 3], 96, 160), ([97, 16, 200], 512, 128),
                                       ([33, 64], 1056, 416), ([2] * 30, 256, 256), ([96, 200], 4096, 64),
                                       ([112, 111, 5, 0, 700, 256], 352, 224), ([300, 0, 1000, 31], 2048, 96),
                                       ([129], 512, 32), ([600, 400], 96, 320)])
def test_swiglu_product_quantises_h(B, pairing, fmt, sizes, K, I):
    rng = np.random.default_rng(K + I + fmt)
    E, rows, blk = len(sizes), sum(sizes), BLOCK[fmt]
    ac, asc = random_operand(rng, (rows,), K, fmt)
    wc, wsc = random_operand(rng, (E, 2 * I), K, fmt)
    a2, w2, h2 = np.float32(0.05), (rng.random(E) * 0.05 + 0.01).astype(np.float32), np.float32(0.02)
    ws = status_ws()
    hc, hs = B.fp4_grouped_gemm_swiglu(dev(ac), dev(asc), dev(wc), dev(wsc), dev(np.array(sizes, np.int32)), fmt,
                                       act_scale_2=scale1(a2), weight_scale_2=dev(w2), h_scale_2=scale1(h2),
                                       workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    hc, hs = hc.cpu().numpy(), hs.cpu().numpy()
    g = float(h2) if fmt == NV else 1.0
    hq, unit = values(hc, hs, fmt) * g, np.repeat(scale_values(hs, fmt) * g, blk, axis=1)
    a, r = values(ac, asc, fmt), 0
    for e, n in enumerate(sizes):
        if n == 0:
            continue
        s = float(a2 * w2[e]) if fmt == NV else 1.0
        h, tau = swiglu_reference(a[r:r + n], values(wc[e], wsc[e], fmt), I, s)
        top = np.abs(h).reshape(n, -1, blk).max(-1)
        ttop = tau.reshape(n, -1, blk).max(-1)
        lo, hi = (quantise_byte(np.maximum(top - ttop, 0), fmt, h2), quantise_byte(top + ttop, fmt, h2))
        assert np.all((hs[r:r + n] >= lo) & (hs[r:r + n] <= hi)), e
        u = unit[r:r + n]
        with np.errstate(divide="ignore", invalid="ignore"):
            d = np.where(u > 0, u * nearest_distance(np.abs(h) / u), np.abs(h))
        diff, bound = np.abs(hq[r:r + n] - h), d + 2 * tau
        assert np.all(diff <= bound * (1 + 1e-6)), (e, float((diff - bound).max()))
        r += n


def quantise_byte(a, fmt, g):
    if fmt == MX:
        _, e = np.frexp(a)
        return np.where(a == 0, 0, np.clip(e - 3 + 127, 0, 252))
    return nearest_e4m3(np.minimum(a / (6 * float(g)), 448).astype(np.float32))


def test_swiglu_empty_and_nan(B, pairing):
    rng = np.random.default_rng(12)
    wc, wsc = random_operand(rng, (2, 128), 64, NV)
    ac, asc = random_operand(rng, (6,), 64, NV)
    one = scale1(1)
    kw = dict(act_scale_2=one, weight_scale_2=torch.ones(2, device=DEV))
    hc, hs = B.fp4_grouped_gemm_swiglu(dev(ac[:0]), dev(asc[:0]), dev(wc), dev(wsc), dev(np.zeros(2, np.int32)), NV,
                                       h_scale_2=one, **kw)
    assert hc.shape == (0, 32) and hs.shape == (0, 4)
    for bad in (0.0, float("nan"), -2.0):
        ws = status_ws()
        B.fp4_grouped_gemm_swiglu(dev(ac), dev(asc), dev(wc), dev(wsc), dev(np.array([6, 0], np.int32)), NV,
                                  h_scale_2=scale1(bad), workspace=ws, **kw)
        assert B.read_status(ws) == B.MOE_ERR_DATA


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 64, 32), (53, 3, 9, 288, 160), (20011, 2, 5, 1056, 32)])
def test_layer_equals_its_stages(B, pairing, fmt, T, k, E, H, I):
    rng = np.random.default_rng(T + fmt)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    ids = dev(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32))
    w = torch.rand((T, k), device=DEV)
    w13 = [dev(v) for v in random_operand(rng, (E, 2 * I), H, fmt)] + [torch.rand(E, device=DEV) * 0.1]
    w2 = [dev(v) for v in random_operand(rng, (E, H), I, fmt)] + [torch.rand(E, device=DEV) * 0.1]
    xs2, hs2 = scale1(0.004), scale1(0.01)
    buf = B.LayerBuffersFp4(T, k, E, H, I, fmt, DEV)
    out = B.layer_forward_fp4(x, ids, w, w13, w2, buf, x_scale_2=xs2, h_scale_2=hs2)
    assert B.read_status(buf.workspace) == B.MOE_OK
    gs, _, ss, s2r, _ = B.route_sort(ids, E)
    xc, xs = B.fp4_quantize(x, fmt, row_index=ss, index_div=k, tensor_scale=xs2)
    h = B.fp4_grouped_gemm_swiglu(xc, xs, w13[0], w13[1], gs, fmt, act_scale_2=xs2, weight_scale_2=w13[2],
                                  h_scale_2=hs2)
    y = B.fp4_grouped_gemm(*h, w2[0], w2[1], gs, fmt, act_scale_2=hs2, weight_scale_2=w2[2])
    assert torch.equal(out, B.combine(y, s2r, w))


# ---------------------------------------------------------------- refusals

def test_binding_refuses_what_it_would_misread(B):
    x = torch.zeros((4, 64), device=DEV)
    c, s = B.fp4_quantize(x, MX)
    wc = torch.zeros((2, 8, 32), dtype=torch.uint8, device=DEV)
    wsc = torch.zeros((2, 8, 2), dtype=torch.uint8, device=DEV)
    gs = torch.tensor([4, 0], dtype=torch.int32, device=DEV)
    ok = dict(act_codes=c, act_scales=s, codes=wc, scales=wsc, group_sizes=gs, fmt=MX)
    B.fp4_grouped_gemm(**ok)
    for change in (dict(act_scales=s[:, :1]), dict(codes=wc[:, :, :16]), dict(group_sizes=gs.long()),
                   dict(fmt=7), dict(fmt=NV), dict(scales=wsc.cpu()), dict(out=torch.zeros((4, 8), device=DEV).half())):
        with pytest.raises(ValueError):
            B.fp4_grouped_gemm(**{**ok, **change})
    for bad in (x.half(), x.T, x.cpu()):
        with pytest.raises(ValueError):
            B.fp4_quantize(bad, MX)
    with pytest.raises(B.MoeError):
        B.fp4_quantize(torch.zeros((4, 48), device=DEV), MX,
                       out=(torch.zeros((4, 24), dtype=torch.uint8, device=DEV),
                            torch.zeros((4, 1), dtype=torch.uint8, device=DEV)))
    with pytest.raises(B.MoeError):     # a code buffer off 16 bytes
        flat = torch.zeros(4 * 32 + 16, dtype=torch.uint8, device=DEV)
        B.fp4_grouped_gemm(**{**ok, "act_codes": flat[8:8 + 128].view(4, 32)})
