"""Gradients of the weighted unsort (moe_combine_backward) and of the sort's gather
(moe_gather_backward) against plain forms.

Tolerances, fixed before the first run.  dy: one f32 product, rounded once more for
bf16: exact.  dx: f32 additions in ascending j, rounded once: exact against the same
sums on the CPU, and within (k + 1) 2^-24 sum |a| of 64 bits.  dw: a lane adds N / 32
products by fused multiply-add, the warp joins 32 lanes: (N / 32 + 8) 2^-24 sum |a b|.
"""
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


def routed(B, seed, T, E, k):
    ids = torch.from_numpy(inputs.route_uniform(seed, T, E, k)).to(DEV)
    return B.route_sort(ids, E)[3]


def rand(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


SHAPES = [(1, 4, 1, 1), (1, 8, 6, 40), (5, 8, 2, 33), (37, 16, 3, 4), (64, 64, 6, 1028), (130, 8, 8, 4096), (3, 4, 2, 7)]


@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, F32, BF16), (BF16, BF16, F32), (F32, BF16, BF16)],
                         ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("T,E,k,N", SHAPES)
def test_combine_backward(B, T, E, k, N, types):
    gen = torch.Generator(device=DEV).manual_seed(T + N)
    s2r = routed(B, T, T, E, k)
    w = torch.rand((T, k), generator=gen, device=DEV)
    w.view(-1)[0] = 0.0
    dout, y = rand(gen, (T, N), types[0]), rand(gen, (T * k, N), types[1])
    dy, dw = B.combine_backward(dout, y, s2r, w, dy_dtype=types[2])
    again = B.combine_backward(dout, y, s2r, w, dy_dtype=types[2])
    assert torch.equal(dy, again[0]) and torch.equal(dw, again[1])
    at = s2r.long()
    want = (w[:, :, None] * dout.float()[:, None, :]).view(T * k, N).to(types[2])
    assert torch.equal(dy[at], want)
    a, b = dout.double()[:, None, :], y.double()[at].view(T, k, N)
    ref, mag = (a * b).sum(-1), (a * b).abs().sum(-1)
    assert bool(((dw.double() - ref).abs() <= (N / 32 + 8) * 2.0 ** -24 * mag).all())


@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, BF16, BF16)], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,N", [(200, 8, 3, 72), (9, 8, 4, 12), (33, 8, 2, 3), (3, 4, 2, 1024), (16, 8, 8, 4096),
                                     (64, 8, 6, 516), (5, 8, 2, 131)])
def test_combine_backward_short_rows_and_few_slots(B, T, E, k, N, types):
    """Fewer threads a slot than a warp, and a whole block, with slots that have no row.
    dw: a lane adds up to max(8, N / 32) products and at most 8 + 5 joins follow."""
    gen = torch.Generator(device=DEV).manual_seed(T + N)
    ids = inputs.route_uniform(T, T, E, k)
    ids.reshape(-1)[1::5] = -1
    s2r = B.route_sort(torch.from_numpy(ids).to(DEV), E)[3]
    w = torch.rand((T, k), generator=gen, device=DEV)
    dout, y = rand(gen, (T, N), types[0]), rand(gen, (T * k, N), types[1])
    out = torch.full((T * k, N), 7.0, dtype=types[2], device=DEV)
    dw = torch.full((T, k), 7.0, device=DEV)
    dy, _ = B.combine_backward(dout, y, s2r, w, out=(out, dw))
    on, at = s2r >= 0, s2r.clamp_min(0).long()
    want = torch.full_like(out, 7.0)
    want[at[on]] = (w[:, :, None] * dout.float()[:, None, :]).view(T * k, N).to(types[2])[on]
    assert torch.equal(dy, want)
    prod = dout.double()[:, None, :] * y.double()[at].view(T, k, N) * on.view(T, k, 1)
    ref, mag = prod.sum(-1), prod.abs().sum(-1)
    assert bool(((dw.double() - ref).abs() <= (max(8, N / 32) + 13) * 2.0 ** -24 * mag).all())
    assert torch.equal(dw, B.combine_backward(dout, y, s2r, w)[1])


@pytest.mark.parametrize("src,dst", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("T,E,k,N", SHAPES)
def test_gather_backward(B, T, E, k, N, src, dst):
    gen = torch.Generator(device=DEV).manual_seed(T + N)
    s2r = routed(B, T, T, E, k)
    g = rand(gen, (T * k, N), src)
    dx = B.gather_backward(g, s2r, k, out=torch.empty((T, N), dtype=dst, device=DEV))
    rows = g.float()[s2r.long()].view(T, k, N)
    acc = torch.zeros((T, N), device=DEV)
    for j in range(k):
        acc = acc + rows[:, j]
    assert torch.equal(dx, acc.to(dst))
    if dst == F32:
        ref, mag = rows.double().sum(1), rows.double().abs().sum(1)
        assert bool(((dx.double() - ref).abs() <= (k + 1) * 2.0 ** -24 * mag).all())


def test_dropped_slots(B):
    """Slots without a row (ids out of range): weight gradient 0, no row read or
    written, nothing added to dx."""
    T, k, N, E = 9, 4, 24, 6
    ids = torch.from_numpy(inputs.route_uniform(3, T, E, k)).to(DEV)
    ids[0] = -1                                   # a token without any row
    ids[3, 1] = E
    ids[8, 3] = 2 ** 31 - 1
    _, off, _, s2r, _ = B.route_sort(ids, E)
    valid = int(off[E])
    assert valid == T * k - 6
    w = torch.rand((T, k), device=DEV)
    dout, y = torch.randn((T, N), device=DEV), torch.randn((T * k, N), device=DEV)
    y[valid:] = float("nan")
    dy = torch.full((T * k, N), 5.0, device=DEV)
    dw = torch.full((T, k), 5.0, device=DEV)
    B.combine_backward(dout, y, s2r, w, out=(dy, dw))
    keep = (s2r >= 0).view(T, k)
    assert bool((dy[valid:] == 5.0).all()) and bool((dw[~keep] == 0).all())
    at = s2r[s2r >= 0].long()
    tok = torch.arange(T, device=DEV)[:, None].expand(T, k)[keep]
    assert torch.equal(dy[at], w[keep][:, None] * dout[tok])
    assert torch.allclose(dw[keep], (dout[tok] * y[at]).sum(1), atol=1e-5)
    dx = B.gather_backward(y, s2r, k)
    assert bool((dx[0] == 0).all()) and not bool(dx.isnan().any())


def test_no_tokens(B):
    z = torch.zeros((0, 8), device=DEV)
    dy, dw = B.combine_backward(z, z, torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros((0, 2), device=DEV))
    assert dy.shape == (0, 8) and dw.shape == (0, 2)
    assert B.gather_backward(z, torch.zeros(0, dtype=torch.int32, device=DEV), 2).shape == (0, 8)


def test_gradients_against_differences_of_the_forward(B):
    """combine is linear in y and in w, so a difference of its f32 outputs with a step of
    one is the derivative up to f32 rounding: (k + 2) 2^-24 of the terms' magnitudes,
    summed over N."""
    T, k, N, E = 6, 3, 16, 5
    s2r = routed(B, 1, T, E, k)
    gen = torch.Generator(device=DEV).manual_seed(2)
    w, y, dout = torch.rand((T, k), generator=gen, device=DEV), rand(gen, (T * k, N), F32), rand(gen, (T, N), F32)
    dy, dw = B.combine_backward(dout, y, s2r, w)
    loss = lambda y, w: float((B.combine(y, s2r, w).double() * dout.double()).sum())  # noqa: E731
    base = loss(y, w)
    tol = 64 * (k + 2) * 2.0 ** -24 * float((dout.abs().max() * (1 + y.abs().max())) * N)
    for t, j in ((0, 0), (5, 2), (3, 1)):
        w1 = w.clone()
        w1[t, j] += 1
        assert abs(loss(y, w1) - base - float(dw[t, j])) <= tol
        r, n = int(s2r[t * k + j]), 7
        y1 = y.clone()
        y1[r, n] += 1
        assert abs(loss(y1, w) - base - float(dy[r, n])) <= tol


def test_rows_past_32_bits(B):
    """T*k*N over 2^31 elements, bf16: the last token's rows."""
    T, k, N = 2050, 2, 524800
    s2r = torch.randperm(T * k, device=DEV).to(torch.int32)
    w = torch.rand((T, k), device=DEV)
    dout = torch.randn((T, 64), device=DEV).to(BF16).repeat(1, N // 64)
    y = torch.empty((T * k, N), dtype=BF16, device=DEV).fill_(0.5)
    dy, dw = B.combine_backward(dout, y, s2r, w)
    for t in (0, T - 1):
        at = s2r[t * k:t * k + k].long()
        assert torch.equal(dy[at], (w[t][:, None] * dout[t].float()).to(BF16))
        ref, mag = 0.5 * dout[t].double().sum(), 0.5 * dout[t].double().abs().sum()
        assert bool(((dw[t].double() - ref).abs() <= (N / 32 + 8) * 2.0 ** -24 * mag).all())
    dx = B.gather_backward(dy, s2r, k)
    at = s2r[(T - 1) * k:].long()
    assert torch.equal(dx[T - 1], (dy[at[0]].float() + dy[at[1]].float()).to(BF16))


def test_refusals(B):
    s2r = torch.zeros(6, dtype=torch.int32, device=DEV)
    w, d, y = torch.zeros((3, 2), device=DEV), torch.zeros((3, 8), device=DEV), torch.zeros((6, 8), device=DEV)
    for bad in (dict(dout=d.half()), dict(y=y[:5]), dict(s2r=s2r.long()), dict(w=w.double()), dict(dout=d[:, ::2]),
                dict(y=y.cpu())):
        a = {**dict(dout=d, y=y, s2r=s2r, w=w), **bad}
        with pytest.raises(ValueError):
            B.combine_backward(a["dout"], a["y"], a["s2r"], a["w"])
    for k in (0, 4):
        with pytest.raises(ValueError):
            B.gather_backward(y, s2r, k)
    with pytest.raises(B.MoeError):               # rows off 16 bytes
        flat = torch.zeros(6 * 8 + 4, device=DEV)
        B.gather_backward(flat[1:49].view(6, 8), s2r, 2)
