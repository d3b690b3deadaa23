"""The CTA-pair kernel of the W4A4 products, whose odd CTA hands its scale columns over through
a relay: every stage's scales reach the sums of that stage, in both CTAs' rows.

Tolerance: |gpu - exact| <= 1e-5 * sum_k |a w| + 1e-6, the library's bound for f32 sums.
"""
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


@pytest.fixture
def pairs(B):
    B.set_gemm_pairing(B.MOE_PAIRING_ON)
    yield
    B.set_gemm_pairing(B.MOE_PAIRING_AUTO)


def e2m1():
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    return torch.cat([m, -m])


def scale_table(fmt):
    b = torch.arange(256, device=DEV)
    if fmt == MX:
        return torch.ldexp(torch.ones(256, dtype=torch.float64, device=DEV), b - 127)
    e, m = b >> 3 & 15, (b & 7).double()
    return torch.where(e == 0, m / 512, torch.ldexp(1 + m / 8, e - 7))


def values(codes, scales, fmt):
    """Codes uint8 [R, K/2] and block scales -> float64 [R, K]."""
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(1).long()
    return e2m1()[nib] * scale_table(fmt)[scales.long()].repeat_interleave(BLOCK[fmt], dim=1)


def codes_of(gen, shape, K):
    return torch.randint(0, 256, (*shape, K // 2), generator=gen, device=DEV, dtype=torch.uint8)


def scale1(v):
    return torch.full((1,), float(v), device=DEV)


@pytest.mark.parametrize("fmt", [MX, NV], ids=["mx", "nv"])
@pytest.mark.parametrize("K", [8192, 4096 + 96])
def test_scales_of_every_stage_reach_its_sums(B, pairs, fmt, K):
    """Stage s (256 k) of a row has scales that no other stage nor row near it has: a column
    left from another stage would be wrong by a power of two at least."""
    gen = torch.Generator(device=DEV).manual_seed(K + fmt)
    sizes, N = [1024, 0, 700, 513], 384
    rows, E = sum(sizes), len(sizes)
    per, stage = K // BLOCK[fmt], 256 // BLOCK[fmt]

    def scales(shape):
        s = torch.arange(per, device=DEV) // stage
        r = torch.arange(int(np.prod(shape)), device=DEV)[:, None]
        step = (7 * s[None, :] + 3 * r) % 9                      # 2^-4 .. 2^4 in turn
        b = 123 + step - 4 if fmt == MX else (7 + step - 4) << 3
        return b.to(torch.uint8).view(*shape, per)

    ac, asc = codes_of(gen, (rows,), K), scales((rows,))
    wc, wsc = codes_of(gen, (E, N), K), scales((E, N))
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    kw = dict(act_scale_2=scale1(1), weight_scale_2=torch.ones(E, device=DEV), workspace=ws)
    torch.cuda.synchronize()
    out = B.fp4_grouped_gemm(ac, asc, wc, wsc, gs, fmt, **kw)
    assert B.read_status(ws) == B.MOE_OK
    r = 0
    for e, n in enumerate(sizes):
        if n:
            a, w = values(ac[r:r + n], asc[r:r + n], fmt), values(wc[e], wsc[e], fmt)
            ref, mag = a @ w.T, a.abs() @ w.abs().T
            assert bool(((out[r:r + n].double() - ref).abs() <= 1e-5 * mag + 1e-6).all()), e
        r += n
    for _ in range(30):
        assert torch.equal(out, B.fp4_grouped_gemm(ac, asc, wc, wsc, gs, fmt, **kw))
