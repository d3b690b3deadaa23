"""What the W4A4 products report and how they read scales, in both kernels and by both ways that
scales take into them: bytes the formats do not allow, scale tensors at any address, blocks of
h that are not finite; and the products over 256 experts at a layer's sizes.

Exact comparisons are between runs of the same sums; tolerances are those of the products'
and the SwiGLU product's tests.
"""
import numpy as np
import pytest
import torch

from parity_bounds import SILU_SLOPE_MAX
from test_gpu_fp4 import (BLOCK, MX, NV, dev, nearest_distance, quantise_byte, random_operand, scale1, scale_values,
                          status_ws, values)
from test_gpu_fp4_pairs import values as gpu_values

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = dict(argvalues=[MX, NV], ids=["mx", "nv"])


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


@pytest.fixture(params=["off", "on"])
def pairing(B, request):
    """Long bands in the short bands' kernel, or in CTA pairs."""
    B.set_gemm_pairing(B.MOE_PAIRING_ON if request.param == "on" else B.MOE_PAIRING_OFF)
    yield
    B.set_gemm_pairing(B.MOE_PAIRING_AUTO)


# ------------------------------------------------------ bytes not allowed

# K of whole 16-byte scale rows (copied by TMA) and of others (by threads).
K_OF = {MX: (512, 1024, 288), NV: (256, 512, 288)}
ROWS, COLS = (0, 29, 30, 63, 95, 126, 158, 190, 222, 254, 286, 329), (0, 31, 63, 95, 100, 127, 130, 159, 191, 192, 223)


@pytest.mark.parametrize("fmt", **FORMATS)
@pytest.mark.parametrize("which", [0, 1, 2], ids=["one_group", "groups", "shifted"])
@pytest.mark.parametrize("side", ["act", "weight"])
def test_bad_scales_are_reported_wherever_they_are(B, pairing, fmt, which, side):
    """A byte in every row group and every word in turn, in a short and a long band: reported,
    and only its row or column differs from a clean run."""
    rng = np.random.default_rng(100 + fmt)
    K, N, sizes = K_OF[fmt][which], 256, [30, 300]
    per = K // BLOCK[fmt]
    ac, asc = (dev(v) for v in random_operand(rng, (sum(sizes),), K, fmt))
    wc, wsc = (dev(v) for v in random_operand(rng, (2, N), K, fmt))
    gs = dev(np.array(sizes, np.int32))
    kw = dict(act_scale_2=scale1(1), weight_scale_2=torch.ones(2, device=DEV))
    clean = B.fp4_grouped_gemm(ac, asc, wc, wsc, gs, fmt, **kw)
    h2 = scale1(0.02)
    h_clean = B.fp4_grouped_gemm_swiglu(ac, asc, wc, wsc, gs, fmt, h_scale_2=h2, **kw)
    nan_bytes = [255] if fmt == MX else [0x7F, 0xFF, 0x80]
    for i, at in enumerate(ROWS if side == "act" else COLS):
        e = i % 2
        where = (at,) if side == "act" else (e, at)
        s = (asc if side == "act" else wsc).clone()
        s[where][(5 * i) % per] = nan_bytes[i % len(nan_bytes)]
        pair = (s, wsc) if side == "act" else (asc, s)
        ws = status_ws()
        out = B.fp4_grouped_gemm(ac, pair[0], wc, pair[1], gs, fmt, workspace=ws, **kw)
        assert B.read_status(ws) == B.MOE_ERR_DATA, (at, i)
        ws = status_ws()
        hc, hs = B.fp4_grouped_gemm_swiglu(ac, pair[0], wc, pair[1], gs, fmt, h_scale_2=h2, workspace=ws, **kw)
        assert B.read_status(ws) == B.MOE_ERR_DATA, (at, i)
        keep = torch.ones((sum(sizes), N), dtype=torch.bool, device=DEV)
        blocks = torch.ones((sum(sizes), N // 2 // BLOCK[fmt]), dtype=torch.bool, device=DEV)
        if side == "act":
            keep[at], blocks[at] = False, False
        else:
            rows = slice(0, 30) if e == 0 else slice(30, None)
            keep[rows, at], blocks[rows, at % (N // 2) // BLOCK[fmt]] = False, False
        assert torch.equal(out[keep], clean[keep])
        assert torch.equal(hs[blocks], h_clean[1][blocks])
        per_code = blocks.repeat_interleave(BLOCK[fmt] // 2, dim=1)
        assert torch.equal(hc[per_code], h_clean[0][per_code])


# ------------------------------------------------------ scale addresses

@pytest.mark.parametrize("fmt", **FORMATS)
@pytest.mark.parametrize("K", [512, 320])
@pytest.mark.parametrize("offset", [1, 4, 8, 15])
def test_scale_tensors_at_any_address(B, pairing, fmt, K, offset):
    """Scales off 16 bytes, one tensor or both: the bits that aligned ones give."""
    rng = np.random.default_rng(K + offset)
    N, sizes = 448, [300, 0, 40, 113, 1]
    ac, asc = random_operand(rng, (sum(sizes),), K, fmt)
    wc, wsc = random_operand(rng, (len(sizes), N), K, fmt)
    gs = dev(np.array(sizes, np.int32))
    kw = dict(act_scale_2=scale1(0.5), weight_scale_2=torch.full((len(sizes),), 0.25, device=DEV))
    h2 = scale1(0.02)

    def at(s, off):
        buf = torch.full((s.size + 64,), 255, dtype=torch.uint8, device=DEV)
        v = buf[off:off + s.size].view(s.shape)
        v.copy_(dev(s))
        return v

    def run(a_off, w_off):
        ws = status_ws()
        ops = (dev(ac), at(asc, a_off), dev(wc), at(wsc, w_off), gs, fmt)
        out = B.fp4_grouped_gemm(*ops, workspace=ws, **kw)
        h = B.fp4_grouped_gemm_swiglu(*ops, h_scale_2=h2, workspace=ws, **kw)
        assert B.read_status(ws) == B.MOE_OK        # nor are the bytes around the tensors looked at
        return (out, *h)

    want = run(0, 0)
    for offsets in ((offset, offset), (offset, 0), (0, offset)):
        assert all(torch.equal(a, b) for a, b in zip(want, run(*offsets))), offsets


# ------------------------------------------------------ h that is not finite

@pytest.mark.parametrize("fmt", **FORMATS)
@pytest.mark.parametrize("K", [256, 96])
def test_blocks_of_h_that_are_not_finite(B, pairing, fmt, K):
    """Gate and up sums that overflow: +inf in block 0 (silu(inf) inf), zeros in block 1, NaN in
    block 2 (silu(-inf) = -inf * 0), in a row of a short band and two of a long one.  Those
    blocks get the NaN scale and zero codes; every other block is zero."""
    I, sizes = 96, [20, 300]
    rows, blk = sum(sizes), BLOCK[fmt]
    hot = [7, 20 + 5, 20 + 299]
    ac = torch.zeros((rows, K // 2), dtype=torch.uint8, device=DEV)
    ac[hot] = 0x77                                       # 6.0 throughout
    asc = torch.full((rows, K // blk), 254 if fmt == MX else 0x7E, dtype=torch.uint8, device=DEV)
    wc = torch.zeros((2, 2 * I, K // 2), dtype=torch.uint8, device=DEV)
    wc[:, 0:32], wc[:, I:I + 32] = 0x77, 0x77
    wc[:, 64:96], wc[:, I + 64:I + 96] = 0xFF, 0x77      # gate -6.0, up 6.0
    wsc = torch.full((2, 2 * I, K // blk), 127 if fmt == MX else 0x38, dtype=torch.uint8, device=DEV)
    ws = status_ws()
    hc, hs = B.fp4_grouped_gemm_swiglu(ac, asc, wc, wsc, dev(np.array(sizes, np.int32)), fmt, act_scale_2=scale1(3e38),
                                       weight_scale_2=torch.ones(2, device=DEV), h_scale_2=scale1(0.5), workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    want = torch.zeros((rows, I // blk), dtype=torch.uint8, device=DEV)
    nan = 255 if fmt == MX else 0x7F
    for r in hot:
        want[r, :32 // blk], want[r, 64 // blk:] = nan, nan
    assert torch.equal(hs, want)
    assert int(hc.max()) == 0
    # and the next product reports them
    w2, w2s = torch.zeros((2, 32, I // 2), dtype=torch.uint8, device=DEV), torch.zeros((2, 32, I // blk),
                                                                                     dtype=torch.uint8, device=DEV)
    B.fp4_grouped_gemm(hc, hs, w2, w2s, dev(np.array(sizes, np.int32)), fmt, act_scale_2=scale1(1),
                       weight_scale_2=torch.ones(2, device=DEV), workspace=ws)
    assert B.read_status(ws) == B.MOE_ERR_DATA


# ------------------------------------------------------ 256 experts, layer sizes

def spread(rng, T, E, k, zipf):
    """k distinct experts a token: uniform, or Zipf(1.1) with the last 19 unused."""
    logp = -1.1 * np.log(np.arange(1, E + 1)) if zipf else np.zeros(E)
    if zipf:
        logp[E - 19:] = -1e9
    key = logp[rng.permutation(E)] - np.log(-np.log(rng.random((T, E)).clip(1e-12, 1 - 1e-12)))
    return np.bincount(np.argsort(-key, axis=1)[:, :k].ravel(), minlength=E)


@pytest.mark.parametrize("fmt", **FORMATS)
@pytest.mark.parametrize("T,zipf", [(64, False), (4096, True), (8192, False)])
def test_256_experts_at_layer_sizes(B, fmt, T, zipf):
    """w13 with SwiGLU (K = 4,096, I = 2,048) and w2 (K = 2,048, N = 4,096): the first, the last
    and one more row of every band, all columns."""
    rng = np.random.default_rng(T + fmt)
    gen = torch.Generator(device=DEV).manual_seed(T + fmt)
    E, k, H, I, blk = 256, 6, 4096, 2048, BLOCK[fmt]
    sizes = spread(rng, T, E, k, zipf)
    rows = int(sizes.sum())
    assert rows == T * k and sizes.min() < sizes.max()
    lo, hi = (119, 124) if fmt == MX else (0, 0x50)

    def operand(*shape, K):
        return (torch.randint(0, 256, (*shape, K // 2), generator=gen, device=DEV, dtype=torch.uint8),
                torch.randint(lo, hi, (*shape, K // blk), generator=gen, device=DEV, dtype=torch.uint8))

    gs, ws, h2 = dev(sizes.astype(np.int32)), status_ws(), np.float32(0.02)
    a, w13, w2 = operand(rows, K=H), operand(E, 2 * I, K=H), operand(E, H, K=I)
    g13 = torch.full((E,), 0.01, device=DEV)
    hc, hs = B.fp4_grouped_gemm_swiglu(*a, *w13, gs, fmt, act_scale_2=scale1(0.01), weight_scale_2=g13,
                                       h_scale_2=scale1(h2), workspace=ws)
    y = B.fp4_grouped_gemm(hc, hs, *w2, gs, fmt, act_scale_2=scale1(h2), weight_scale_2=g13, workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    s13 = float(np.float32(0.01)) ** 2 if fmt == NV else 1.0
    s2 = float(h2) * float(np.float32(0.01)) if fmt == NV else 1.0
    off = np.concatenate([[0], np.cumsum(sizes)])
    cpu = lambda t: t.cpu().numpy()  # noqa: E731
    for e in np.nonzero(sizes)[0]:
        n = sizes[e]
        r = off[e] + np.unique([0, n - 1, int(rng.integers(n))])
        at = dev(r)
        h, tau = swiglu_reference(gpu_values(a[0][at], a[1][at], fmt), gpu_values(w13[0][e], w13[1][e], fmt), I, s13)
        got = cpu(hs[at])
        hv, unit = values(cpu(hc[at]), got, fmt), np.repeat(scale_values(got, fmt), blk, axis=1)
        g = float(h2) if fmt == NV else 1.0
        hq, unit = hv * g, unit * g
        top, ttop = np.abs(h).reshape(len(r), -1, blk).max(-1), tau.reshape(len(r), -1, blk).max(-1)
        assert np.all((got >= quantise_byte(np.maximum(top - ttop, 0), fmt, h2)) &
                      (got <= quantise_byte(top + ttop, fmt, h2))), e
        with np.errstate(divide="ignore", invalid="ignore"):
            d = np.where(unit > 0, unit * nearest_distance(np.abs(h) / unit), np.abs(h))
        assert np.all(np.abs(hq - h) <= (d + 2 * tau) * (1 + 1e-6)), e
        w, hv = gpu_values(w2[0][e], w2[1][e], fmt), dev(hv)
        ref, mag = hv @ w.T * s2, hv.abs() @ w.abs().T * s2
        assert bool(((y[at].double() - ref).abs() <= 1e-5 * mag + 1e-6).all()), e


def swiglu_reference(a, w, I, s):
    """h in 64 bits and the f32 error that its rounding may add to: the sums' bounds, and of silu
    (1.25 |g| + 10) 2^-24 (the exponent is rounded once), a few ulps more for the product."""
    y, mag = (a @ w.T * s).cpu().numpy(), (a.abs() @ w.abs().T * s).cpu().numpy()
    g, u = y[:, :I], y[:, I:]
    tg, tu = 1e-5 * mag[:, :I] + 1e-6, 1e-5 * mag[:, I:] + 1e-6
    silu = g / (1 + np.exp(-g))
    h = silu * u
    return h, SILU_SLOPE_MAX * tg * (np.abs(u) + tu) + np.abs(silu) * tu + (1.25 * np.abs(g) + 16) * 2.0 ** -24 * np.abs(h)
