"""Exact zeros in the gradient norm: the router rows of experts that nobody chose, embedding rows
outside of the batch; and elements so small that f32 does not hold their squares.  Element by element
in f64 a list of either took 7 (f32) to 13 (bf16) times as long as others."""
import math

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


def micros(f):
    """The fastest of several batches of calls, one after another."""
    best = math.inf
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 5 * 1e3)
    return best


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_are_as_fast_as_other_gradients(B, dtype):
    """Half a gigabyte: all zeros, every second row, half of each cache line, and elements of 2^-60,
    against ordinary ones."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = 1 << (14 if dtype == torch.float32 else 15)
    x = torch.randn((rows, 8192), generator=g, device="cuda").to(dtype)
    ws = torch.zeros(B.MOE_GRAD_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")
    ordinary = micros(lambda: B.grad_norm([x], norm=norm, workspace=ws))
    some = x.clone()
    some[::2] = 0
    few = x.clone()
    few.view(-1, 64)[:, :32] = 0
    for y in (torch.zeros_like(x), some, few, x * 2.0 ** -60):
        assert micros(lambda: B.grad_norm([y], norm=norm, workspace=ws)) < 3 * ordinary


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("power", [-133, -126, -100, -80, -46, -30])
def test_tiny_elements_among_zeros(B, power, dtype):
    """One element that is not 0 in a group, at any place of it; the norm within 5 2^-24 (f32 sums of
    a group's squares, 4 2^-24, and one rounding), and half a step of 2^-149."""
    n = 3 * 4 * 512 * 8 + 5
    for at in (0, 1, 7, 8, 31, 512 * 8, 2 * 512 * 8 + 3, n - 6, n - 1):
        for value in (1.0, -1.5):
            x = torch.zeros(n, device="cuda", dtype=dtype)
            x[at] = value * 2.0 ** power
            x[n // 2] = -0.0
            want = float(x.double().norm())
            assert want > 0
            assert abs(float(B.grad_norm([x])) - want) <= 5 * 2.0 ** -24 * want + 2.0 ** -150
            keep = x.clone()
            norm = B.clip_grads([x], 1.0)
            assert float(norm) <= 1 and torch.equal(x, keep)


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_one_element_that_is_not_finite_among_zeros(B, value):
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(100001, device="cuda", dtype=dtype)
        x[54321] = value
        norm = float(B.grad_norm([x]))
        assert math.isnan(norm) if math.isnan(value) else math.isinf(norm)
