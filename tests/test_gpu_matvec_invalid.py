"""Few-row products in which many rows name no expert: their outputs are zeros, the others' what
they are without them, and the whole GPU writes them."""
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


def weights(g, E, N, K, fmt):
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == 0:
        return codes, torch.randint(118, 124, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8), None
    scales = torch.randint(0x28, 0x41, (E, N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales, torch.rand((E,), generator=g, device="cuda") + 0.5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("rows,N", [(1, 1), (3, 1023), (20, 1025), (33, 7), (100, 3001), (512, 1100)])
def test_rows_without_an_expert_are_zeros(B, rows, N, fmt, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    E, K = 5, 96
    w = weights(g, E, N, K, fmt)
    x = torch.randn((rows, K), generator=g, device="cuda").bfloat16()
    for some in (0.0, 0.5, 0.97):                                 # how many rows have an expert
        ids = torch.randint(0, E, (rows,), generator=g, device="cuda", dtype=torch.int32)
        bad = torch.rand((rows,), generator=g, device="cuda") >= some
        bad[rows // 2] = True
        named = torch.where(bad, torch.where(ids % 2 == 0, -1 - ids, E + ids * 1000003), ids)
        buf = torch.full((rows + 2, N), 7.0, device="cuda", dtype=dtype)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        out = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=named, weight_scale_2=w[2], out=buf[1:-1], workspace=ws)
        assert B.read_status(ws) == B.MOE_ERR_DATA
        assert bool((out[bad] == 0).all()) and bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())
        want = x.double() @ torch.zeros((K, N), dtype=torch.float64, device="cuda")
        for e in range(E):
            here = (ids == e) & ~bad
            want[here] = x[here].double() @ dense(w, e, fmt).T
        tol = 1e-5 * 40 * K + (want.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0)
        assert bool(((out.double() - want).abs() <= tol).all())


def dense(w, e, fmt):
    codes, scales, ws2 = w
    b = codes[e].long()
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    table = torch.tensor(mags + [-m for m in mags], dtype=torch.float64, device="cuda")
    v = torch.stack([table[b & 15], table[b >> 4]], dim=-1).flatten(-2)
    if fmt == 0:
        return v * torch.pow(torch.full((), 2.0, dtype=torch.float64, device="cuda"), scales[e].double() - 127).repeat_interleave(32, -1)
    return v * scales[e].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * ws2[e].double()


def micros(f):
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


def test_many_rows_without_an_expert_cost_no_more_than_with_one(B):
    """512 rows of 32,768 columns, 67 MB of zeros, against the same rows with weights to read."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, E, N, K = 512, 512, 32768, 64
    w = weights(g, E, N, K, 0)
    x = torch.randn((rows, K), generator=g, device="cuda").bfloat16()
    out = torch.empty((rows, N), device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ids = torch.arange(rows, device="cuda", dtype=torch.int32)
    none = torch.full_like(ids, -1)
    call = lambda i: lambda: B.fp4_matvec(x, w[0], w[1], 0, row_expert=i, out=out, workspace=ws)  # noqa: E731
    assert micros(call(none)) < micros(call(ids))
    assert bool((out != 0).any())
    call(none)()
    assert bool((out == 0).all())
