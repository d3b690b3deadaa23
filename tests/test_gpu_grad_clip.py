"""Global gradient norm and clipping against the formulas in 64 bits.

The norm: squares of a thread's elements are summed in f32, four in a row and three sums
deep (a relative error of at most 7 2^-24, of either sign), the rest in f32 pairs and f64,
and the root halves it: 4 2^-24 is a bound, rounding to f32 adds 2^-24.  A clipped element: the scale rounded to f32, one f32
product, one rounding to the type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
NORM = 5 * 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


def make(g, sizes, dtype, std=1.0):
    pick = {"f32": lambda i: torch.float32, "bf16": lambda i: torch.bfloat16,
            "mixed": lambda i: (torch.float32, torch.bfloat16)[i % 2]}[dtype]
    return [(torch.randn((n,), generator=g, device="cuda") * std).to(pick(i)) for i, n in enumerate(sizes)]


def norm64(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def check(outs, grads, scale):
    for o, x in zip(outs, grads):
        want = x.double() * scale
        tiny = 2.0 ** -149 if x.dtype == torch.float32 else 2.0 ** -133
        rel = half_step(o) + (2 * 2.0 ** -24 + NORM if o.dtype == torch.float32 else NORM + 4 * 2.0 ** -24)
        assert bool(((o.double() - want).abs() <= want.abs() * rel + tiny).all())


LISTS = [[1], [7], [8], [1, 1, 1], [0, 5, 0], [2048, 2049, 2047], [16384 * 3 + 5], [100003, 17, 65536, 3], [513 * 32, 32, 513],
         [11] * 17, [3] * 700, [1 << 22]]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clip(B, sizes, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(sizes))
    grads = make(g, sizes, dtype)
    n = norm64(grads)
    assert abs(float(B.grad_norm(grads)) - n) <= NORM * n
    for factor in (0.25, 4.0):
        outs = [torch.empty_like(t) for t in grads]
        norm = B.clip_grads(grads, factor * n, out=outs)
        assert abs(float(norm) - n) <= NORM * n
        scale = min(1.0, factor * n / (n + 1e-6))
        check(outs, grads, scale)
        if factor > 1:
            assert all(torch.equal(a, b) for a, b in zip(outs, grads))
    again = [t.clone() for t in grads]
    B.clip_grads(again, 0.25 * n)
    outs = [torch.empty_like(t) for t in grads]
    B.clip_grads(grads, 0.25 * n, out=outs)
    assert all(torch.equal(a, b) for a, b in zip(again, outs))                    # in place, the same bits
    assert torch.equal(B.grad_norm(grads), B.grad_norm(grads))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 3), (1, 0), (0, 5), (2, 7)])
def test_any_address(B, a, b, dtype):
    g = torch.Generator(device="cuda").manual_seed(9)
    n = 50001
    src = torch.randn((n + 16,), generator=g, device="cuda").to(dtype)
    dst = torch.full((n + 16,), 7.0, device="cuda").to(dtype)
    x, o = src[a:a + n], dst[b:b + n]
    m = norm64([x])
    B.clip_grads([x], 0.5 * m, out=[o])
    check([o], [x], 0.5 * m / (m + 1e-6))
    assert bool((dst[:b] == 7).all()) and bool((dst[b + n:] == 7).all())


@pytest.mark.parametrize("power", [-140, -126, -100, -70, -40, 30, 62, 100, 120])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_any_magnitude(B, power, dtype):
    """Squares that f32 cannot hold, alone and beside ordinary elements."""
    if dtype == torch.bfloat16 and power == -140:
        power = -130
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (torch.randn((4097,), generator=g, device="cuda").double() * 2.0 ** power).to(dtype)
    n = norm64([x])
    assert abs(float(B.grad_norm([x])) - n) <= NORM * n + 2.0 ** -149
    y = torch.randn((999,), generator=g, device="cuda").to(dtype)
    both = [x, y]
    n = norm64(both)
    assert abs(float(B.grad_norm(both)) - n) <= NORM * n
    out = [torch.empty_like(t) for t in both]
    B.clip_grads(both, 1.0, out=out)
    check(out, both, min(1.0, 1 / (n + 1e-6)))


def test_a_norm_past_f32_still_clips(B):
    x = torch.full((1 << 20,), 3e38, device="cuda")
    out = [torch.empty_like(x)]
    assert math.isinf(float(B.clip_grads([x], 1.0, out=out)))
    check(out, [x], 1.0 / (norm64([x]) + 1e-6))


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_not_finite_scales_nothing(B, value):
    g = torch.Generator(device="cuda").manual_seed(5)
    grads = make(g, [5000, 77], "mixed")
    grads[0][4321] = value
    keep = [t.clone() for t in grads]
    norm = float(B.clip_grads(grads, 0.1))
    assert (math.isnan(norm) if math.isnan(value) else math.isinf(norm) and norm > 0)
    out = [torch.empty_like(t) for t in grads]
    B.clip_grads(grads, 0.1, out=out)
    for a, b, c in zip(grads, keep, out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(c.view(torch.uint8), b.view(torch.uint8))


def test_zeros_and_nothing(B):
    z = [torch.zeros(300, device="cuda"), torch.empty(0, device="cuda")]
    assert float(B.clip_grads(z, 0.0)) == 0.0 and bool((z[0] == 0).all())
    assert float(B.grad_norm([])) == 0.0
    assert float(B.clip_grads([torch.empty(0, device="cuda")], 1.0)) == 0.0
    x = torch.ones(10, device="cuda")
    B.clip_grads([x], 0.0)
    assert bool((x == 0).all())
    x = torch.ones(10, device="cuda")
    B.clip_grads([x], math.inf)
    assert bool((x == 1).all())


def test_overlaps_are_refused(B):
    x = torch.ones(100, device="cuda")
    y = torch.ones(100, device="cuda")
    for grads, out in (([x, x], None), ([x[:50], x[49:]], None), ([x, y], [x, x]), ([x], [y[:99]]),
                       ([x[:50], x[50:]], [x[50:], x[:50]]), ([x[:99]], [x[1:]])):
        with pytest.raises((B.MoeError, ValueError)):
            B.clip_grads(grads, 0.1, out=out)
    assert bool((x == 1).all()) and bool((y == 1).all())
    assert abs(float(B.grad_norm([x, x])) - math.sqrt(200)) < 1e-4        # reading twice is fine
    o = [torch.empty_like(x), torch.empty_like(x)]
    B.clip_grads([x, x], 1.0, out=o)
    assert torch.equal(o[0], o[1])
    B.clip_grads([x[50:], x[:50]], 1.0)                                   # neighbours in either order
    assert bool((x < 1).all())


def test_graphs_and_streams(B):
    g = torch.Generator(device="cuda").manual_seed(6)
    grads = make(g, [30000, 1001, 5], "mixed")
    out = [torch.empty_like(t) for t in grads]
    ws = torch.zeros(B.MOE_GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.clip_grads(grads, 3.0, out=out, norm=norm, workspace=ws)
    for _ in range(3):
        for t in grads:
            t.mul_(1.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        n = norm64(grads)
        assert abs(float(norm) - n) <= NORM * n
        check(out, grads, 3.0 / (n + 1e-6))


def test_two_streams_at_once(B):
    """A workspace each."""
    g = torch.Generator(device="cuda").manual_seed(8)
    grads = [make(g, [50000, 333, 7], "mixed", std) for std in (1.0, 30.0)]
    outs = [[[torch.empty_like(t) for t in grads[i]] for _ in range(8)] for i in range(2)]
    ws = [torch.zeros(B.MOE_GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda") for _ in range(2)]
    norms = [torch.empty(8, device="cuda") for _ in range(2)]
    want = [[torch.empty_like(t) for t in grads[i]] for i in range(2)]
    for i in range(2):
        B.clip_grads(grads[i], 2.0, out=want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for j in range(8):
        for i in range(2):
            B.clip_grads(grads[i], 2.0, out=outs[i][j], norm=norms[i][j:j + 1], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert bool((norms[i] == norms[i][0]).all())
        assert all(torch.equal(a, b) for o in outs[i] for a, b in zip(o, want[i]))


def test_gradients_that_a_kernel_ahead_still_writes(B):
    """Norm and scale in place, over and over: each call sees what the one ahead of it left."""
    x = torch.full((300001,), 8.0, device="cuda")
    for i in range(6):
        n = 8.0 * math.sqrt(300001) * 0.5 ** i
        norm = B.clip_grads([x], 0.5 * n, eps=0.0)
        assert abs(float(norm) - n) <= (i + 1) * NORM * n
    assert bool(((x - 8.0 * 0.5 ** 6).abs() <= 6 * (NORM + 2.0 ** -23) * 8.0 * 0.5 ** 6).all())
