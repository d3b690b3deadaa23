"""Few-row products with 4-bit weights against plain ones in 64 bits.

Tolerance of f32 sums: products are exact, a sum of K of them in f32 in any order is off by
at most about K 2^-24 sum|x w|, in practice sqrt(K) of it; 1e-5 sum|x w| (the grouped
product's own bound) covers K to 16,384 with a margin of 5.  Elements of x below 2^-28 of
their row's largest are rounded to 2^-38 of it, which adds 2^-39 max|x| sum|w|."""
import math

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


def weights(g, E, N, K, fmt, lo=110, hi=130):
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == 0:
        return codes, torch.randint(lo, hi, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8), None
    scales = torch.randint(0, 256, (E, N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    scales[(scales & 0x7F) == 0x7F] = 0x38                       # no NaN; negative ones allowed
    return codes, scales, torch.rand((E,), generator=g, device="cuda") + 0.5


def power2(e):
    """2^e, exact in 64 bits (torch.ldexp of a whole exponent goes through 32)."""
    return torch.tensor([2.0 ** int(i) for i in e.view(-1).tolist()], dtype=torch.float64, device="cuda").view(e.shape)


def dense(w, e, fmt):
    codes, scales, ws2 = w
    b = codes[e].long()
    table = torch.tensor(MAGS + [-m for m in MAGS], dtype=torch.float64, device="cuda")
    v = torch.stack([table[b & 15], table[b >> 4]], dim=-1).flatten(-2)
    if fmt == 0:
        return v * power2(scales[e].double() - 127).repeat_interleave(32, -1)
    return v * scales[e].view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * ws2[e].double()


def check(got, x, w, experts, div, fmt, bf16=False):
    K = x.shape[1]
    for r, e in enumerate(experts):
        xr = x[r // div].double()
        W = dense(w, e, fmt)
        want, mass = W @ xr, W.abs() @ xr.abs()
        tol = 1e-5 * mass + 2.0 ** -39 * xr.abs().max() * W.abs().sum(-1) + 1e-30
        if bf16:
            tol = tol + want.abs() * 2.0 ** -8
        bad = (got[r].double() - want).abs() > tol
        assert not bool(bad.any()), (r, e, K, int(bad.sum()), float((got[r].double() - want).abs().max()))


SHAPES = [  # T, E, k, K, N
    (1, 1, 1, 32, 1), (1, 4, 2, 64, 7), (2, 3, 3, 96, 16), (3, 8, 4, 128, 33), (5, 12, 2, 1056, 713),
    (1, 16, 6, 2048, 100), (8, 16, 6, 160, 50), (16, 2, 2, 512, 40), (9, 1, 1, 2080, 24), (64, 5, 5, 256, 17),
    (17, 1, 1, 4096, 48), (2, 2, 1, 16384, 16), (3, 2, 2, 32768, 9), (512, 7, 1, 64, 20), (1, 1024, 8, 128, 16),
]


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("T,E,k,K,N", SHAPES)
def test_products(B, T, E, k, K, N, fmt):
    g = torch.Generator(device="cuda").manual_seed(T * 131 + K + N)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = weights(g, E, N, K, fmt)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).view(-1)
    ws = B.make_workspace(0, 1, 1)
    out = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, index_div=k, weight_scale_2=w[2], workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    check(out, x, w, ids.tolist(), k, fmt)
    low = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, index_div=k, weight_scale_2=w[2], workspace=ws,
                       out_dtype=torch.bfloat16)
    assert torch.equal(low, out.bfloat16())
    again = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, index_div=k, weight_scale_2=w[2], workspace=ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("T,E,k,K,I", [(1, 1, 1, 32, 1), (1, 8, 6, 2048, 96), (5, 12, 2, 1056, 77), (8, 16, 6, 160, 40),
                                       (33, 3, 2, 544, 13)])
def test_swiglu(B, T, E, k, K, I, fmt):
    """h against the product's own f32 gate and up values: silu is off by a few 2^-24, and
    one rounding to bf16."""
    g = torch.Generator(device="cuda").manual_seed(K + I)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = weights(g, E, 2 * I, K, fmt, 116, 122)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).view(-1)
    ws = B.make_workspace(0, 1, 1)
    args = dict(row_expert=ids, index_div=k, weight_scale_2=w[2], workspace=ws)
    y = B.fp4_matvec(x, w[0], w[1], fmt, **args).double()
    h = B.fp4_matvec_swiglu(x, w[0], w[1], fmt, **args)
    want = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
    assert bool(((h.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-30).all())


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
def test_no_experts_named_is_expert_0(B, fmt):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((11, 416), generator=g, device="cuda").bfloat16()
    w = weights(g, 2, 30, 416, fmt)
    a = B.fp4_matvec(x, w[0], w[1], fmt, weight_scale_2=w[2])
    b = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=torch.zeros(11, dtype=torch.int32, device="cuda"), weight_scale_2=w[2])
    assert torch.equal(a, b)
    check(a, x, w, [0] * 11, 1, fmt)


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_scales_and_rows_at_any_address(B, shift, fmt):
    g = torch.Generator(device="cuda").manual_seed(2)
    K, N, T = 1024, 40, 5
    w = weights(g, 3, N, K, fmt)
    flat = torch.empty(w[1].numel() + 16, dtype=torch.uint8, device="cuda")
    moved = flat[shift:shift + w[1].numel()].view(w[1].shape)
    moved.copy_(w[1])
    big = torch.randn((T, K + 2 * shift + 1), generator=g, device="cuda").bfloat16()
    x = big[:, shift:shift + K]
    ids = torch.tensor([2, 0, 2, 1, 0], dtype=torch.int32, device="cuda")
    got = B.fp4_matvec(x, w[0], moved, fmt, row_expert=ids, weight_scale_2=w[2])
    assert torch.equal(got, B.fp4_matvec(x.contiguous(), w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2]))
    check(got, x, w, ids.tolist(), 1, fmt)


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("power", [-126, -60, -25, 0, 40, 100])
def test_rows_of_any_magnitude(B, power, fmt):
    """Rows from the smallest normal numbers up, wide rows (2^24 between elements), and a zero row."""
    g = torch.Generator(device="cuda").manual_seed(3)
    K, N = 512, 24
    x = torch.randn((4, K), generator=g, device="cuda").double()
    x[1] *= power2(torch.randint(-24, 1, (K,), generator=g, device="cuda"))
    x[2] = 0
    x = (x * 2.0 ** power).bfloat16()
    w = weights(g, 1, N, K, fmt, 118, 124)
    got = B.fp4_matvec(x, w[0], w[1], fmt, weight_scale_2=w[2])
    assert bool((got[2] == 0).all())
    for r in range(4):
        W, xr = dense(w, 0, fmt), x[r].double()
        tol = 1e-5 * (W.abs() @ xr.abs()) + 2.0 ** -39 * xr.abs().max() * W.abs().sum(-1) + 2.0 ** -140
        assert bool(((got[r].double() - W @ xr).abs() <= tol).all())


def test_scale_bytes_at_the_ends(B):
    """Bytes 9 to 252 of MXFP4 with one element a block; 253 and more are reported, and make
    their columns NaN alone."""
    K, N = 32, 253
    codes = torch.zeros((1, N, K // 2), dtype=torch.uint8, device="cuda")
    codes[..., 0] = 2                                            # 1.0 at k = 0
    scales = torch.arange(N, device="cuda").to(torch.uint8).view(1, N, 1)
    x = torch.zeros((1, K), device="cuda").bfloat16()
    x[0, 0] = 1.5
    ws = B.make_workspace(0, 1, 1)
    got = B.fp4_matvec(x, codes, scales, 0, workspace=ws)[0].double()
    want = 1.5 * power2(torch.arange(N, device="cuda") - 127)
    assert torch.equal(got[9:], want[9:])
    assert bool((got[:9] <= want[:9]).all())
    assert B.read_status(ws) == B.MOE_OK
    for b in (253, 254, 255):
        s = scales.clone()
        s[0, 17] = b
        B.clear_status(ws)
        got = B.fp4_matvec(x, codes, s, 0, workspace=ws)[0]
        assert B.read_status(ws) == B.MOE_ERR_DATA
        assert torch.isnan(got).nonzero().view(-1).tolist() == [17]


@pytest.mark.parametrize("K", [64, 1056])
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_nvfp4_nan_scales(B, byte, K):
    g = torch.Generator(device="cuda").manual_seed(5)
    w = weights(g, 2, 33, K, 1)
    x = torch.randn((3, K), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    ws = B.make_workspace(0, 1, 1)
    w[1][1, 5, 0] = byte                                         # of an expert that no row names
    B.fp4_matvec(x, w[0], w[1], 1, row_expert=ids, weight_scale_2=w[2], workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    w[1][0, 32, K // 16 - 1] = byte
    got = B.fp4_matvec(x, w[0], w[1], 1, row_expert=ids, weight_scale_2=w[2], workspace=ws)
    assert B.read_status(ws) == B.MOE_ERR_DATA
    assert bool(torch.isnan(got[:, 32]).all()) and not bool(torch.isnan(got[:, :32]).any())


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
def test_rows_that_are_not_finite_stay_theirs(B, fmt):
    g = torch.Generator(device="cuda").manual_seed(6)
    w = weights(g, 1, 20, 256, fmt)
    x = torch.randn((4, 256), generator=g, device="cuda").bfloat16()
    clean = B.fp4_matvec(x, w[0], w[1], fmt, weight_scale_2=w[2])
    x[1, 3], x[2, 200] = math.nan, math.inf
    got = B.fp4_matvec(x, w[0], w[1], fmt, weight_scale_2=w[2])
    assert bool(torch.isnan(got[1]).all())
    at = dense(w, 0, fmt)[:, 200]
    assert bool((torch.isinf(got[2]) == (at != 0)).all()) and bool((got[2][at > 0] > 0).all())
    assert torch.equal(got[[0, 3]], clean[[0, 3]])


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("bad", [-1, 6, 2 ** 31 - 1])
def test_bad_experts(B, bad, fmt):
    g = torch.Generator(device="cuda").manual_seed(7)
    w = weights(g, 6, 20, 256, fmt)
    x = torch.randn((5, 256), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([5, bad, 3, 5, bad], dtype=torch.int32, device="cuda")
    ws = B.make_workspace(0, 1, 1)
    out = torch.full((6, 20), 7.0, device="cuda")
    B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2], workspace=ws, out=out[:5])
    assert B.read_status(ws) == B.MOE_ERR_DATA
    assert bool((out[[1, 4]] == 0).all()) and bool((out[5] == 7).all())
    check(out[[0, 2, 3]], x[[0, 2, 3]], w, [5, 3, 5], 1, fmt)
    ids[:] = bad
    B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2], workspace=ws, out=out[:5])
    assert bool((out[:5] == 0).all()) and bool((out[5] == 7).all())


def test_no_rows(B):
    g = torch.Generator(device="cuda").manual_seed(8)
    w = weights(g, 2, 16, 64, 0)
    x = torch.empty((0, 64), device="cuda").bfloat16()
    assert B.fp4_matvec(x, w[0], w[1], 0).shape == (0, 16)
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    out = B.layer_decode(x, ids, ids.float(), (torch.zeros((2, 64, 32), dtype=torch.uint8, device="cuda"),
                         torch.zeros((2, 64, 2), dtype=torch.uint8, device="cuda"), None),
                         (torch.zeros((2, 64, 16), dtype=torch.uint8, device="cuda"),
                          torch.zeros((2, 64, 1), dtype=torch.uint8, device="cuda"), None), 0)
    assert out.shape == (0, 64)


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 6, 256, 96), (3, 4, 2, 1056, 544), (8, 16, 4, 512, 256), (40, 6, 3, 64, 32)])
def test_layer(B, T, E, k, H, I, fmt):
    """The layer against its own pieces in 64 bits from the h that it leaves behind, and its
    h against the swiglu product; a slot without an expert adds nothing, whatever its weight."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    w13, w2 = weights(g, E, 2 * I, H, fmt, 116, 122), weights(g, E, H, I, fmt, 116, 122)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    tw = torch.rand((T, k), generator=g, device="cuda")
    ids[0, 1], tw[0, 1] = E, math.nan
    h = torch.empty((T * k, I), device="cuda").bfloat16()
    y2 = torch.empty((T * k, H), device="cuda")
    ws = B.make_workspace(0, 1, 1)
    out = B.layer_decode(x, ids, tw, w13, w2, fmt, h=h, y2=y2, workspace=ws)
    assert B.read_status(ws) == B.MOE_ERR_DATA
    ok = (ids.view(-1) < E).nonzero().view(-1)
    flat = ids.view(-1)
    want_h = B.fp4_matvec_swiglu(x, w13[0], w13[1], fmt, row_expert=flat, index_div=k, weight_scale_2=w13[2])
    assert torch.equal(h[ok], want_h[ok])
    want, mass = torch.zeros((T, H), device="cuda").double(), torch.zeros((T, H), device="cuda").double()
    for r in ok.tolist():
        W = dense(w2, int(flat[r]), fmt) * tw.view(-1)[r].double()
        want[r // k] += W @ h[r].double()
        mass[r // k] += W.abs() @ h[r].double().abs()
    assert bool(((out.double() - want).abs() <= 1e-5 * mass + 1e-30).all())
    assert torch.equal(B.layer_decode(x, ids, tw, w13, w2, fmt, out_dtype=torch.bfloat16), out.bfloat16())


def test_layer_is_the_sorted_layers_result(B):
    """moe_layer_forward on the same input: h is bf16 in both, sums differ in order alone."""
    g = torch.Generator(device="cuda").manual_seed(11)
    T, E, k, H, I = 4, 16, 6, 512, 256
    w13, w2 = weights(g, E, 2 * I, H, 0, 116, 122), weights(g, E, H, I, 0, 116, 122)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    ids, tw = B.topk_gate(torch.randn((T, E), generator=g, device="cuda"), k)
    b = B.LayerBuffers(T, k, E, H, I)
    want = B.layer_forward(x, ids, tw, w13[0], w13[1], w2[0], w2[1], b).double()
    got = B.layer_decode(x, ids, tw, w13, w2, 0).double()
    # an h on a rounding border may go the other way: one bf16 step, 2^-8 of it, on some of I terms
    assert float((got - want).norm() / want.norm()) < 2.0 ** -8


def test_graphs_and_streams(B):
    g = torch.Generator(device="cuda").manual_seed(12)
    w = weights(g, 4, 64, 512, 0)
    x = torch.randn((3, 512), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([3, 1, 3], dtype=torch.int32, device="cuda")
    ws = B.make_workspace(0, 1, 1)
    want = B.fp4_matvec(x, w[0], w[1], 0, row_expert=ids)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        B.fp4_matvec(x, w[0], w[1], 0, row_expert=ids, out=out, workspace=ws)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            B.fp4_matvec(x, w[0], w[1], 0, row_expert=ids, out=out, workspace=ws)
    ids.copy_(torch.tensor([0, 2, 2]))                            # the graph reads the ids when it runs
    x.neg_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, B.fp4_matvec(x, w[0], w[1], 0, row_expert=ids))
    got = B.fp4_matvec(x, w[0], w[1], 0, row_expert=ids, stream=side)
    side.synchronize()
    assert torch.equal(got, out)


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("rows", [9, 20, 33, 100])
def test_many_rows_of_one_expert(B, rows, fmt):
    """More rows of an expert than are taken together, the others' in between."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = weights(g, 40, 36, 288, fmt)
    x = torch.randn((rows, 288), generator=g, device="cuda").bfloat16()
    ids = torch.full((rows,), 7, dtype=torch.int32, device="cuda")
    ids[3], ids[rows - 2] = 39, 0
    got = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2])
    check(got, x, w, ids.tolist(), 1, fmt)
    same = B.fp4_matvec(x[:1].expand(rows, -1), w[0], w[1], fmt, row_expert=torch.full_like(ids, 7), weight_scale_2=w[2])
    assert torch.equal(same, got[:1].expand(rows, -1))


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("K", [32, 256, 1056, 2048, 4608, 12288, 20480])
def test_experts_with_one_to_nine_rows_in_one_call(B, K, fmt):
    """No more rows than experts: experts with one or two rows go their own way, beside others."""
    g = torch.Generator(device="cuda").manual_seed(K)
    w = weights(g, 48, 70, K, fmt)
    counts = {3: 1, 4: 2, 5: 1, 11: 3, 12: 2, 20: 4, 21: 5, 30: 1, 40: 9, 47: 2}
    experts = [e for e, n in counts.items() for _ in range(n)]
    order = torch.randperm(len(experts), generator=g, device="cuda").tolist()
    experts = [experts[i] for i in order]
    x = torch.randn((len(experts), K), generator=g, device="cuda").bfloat16()
    ids = torch.tensor(experts, dtype=torch.int32, device="cuda")
    got = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2])
    check(got, x, w, experts, 1, fmt)
    same = x[:1].expand(len(experts), K).contiguous()
    got = B.fp4_matvec(same, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2])
    for e in counts:
        rows = [r for r, f in enumerate(experts) if f == e]
        assert all(torch.equal(got[r], got[rows[0]]) for r in rows), e


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("rows", [1, 2, 3])
def test_a_row_that_is_not_finite_beside_others_of_its_expert(B, rows, fmt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = weights(g, 9, 40, 512, fmt)
    ids = torch.tensor([4] * rows, dtype=torch.int32, device="cuda")
    x = torch.randn((rows, 512), generator=g, device="cuda").bfloat16()
    clean = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2])
    x[0, 77] = float("inf")
    got = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2])
    assert torch.equal(got[1:], clean[1:])
    at = dense(w, 4, fmt)[:, 77]
    # An infinity times a weight keeps its sign; times 0 it is NaN.
    want = torch.where(at == 0, torch.full_like(at, float("nan")), at.sign() * float("inf"))
    assert torch.equal(got[0].isnan(), want.isnan()) and torch.equal(got[0][at != 0].double(), want[at != 0])


@pytest.mark.parametrize("rows", [1, 2, 3])
@pytest.mark.parametrize("fmt,byte", [(0, 253), (0, 255), (1, 0x7F), (1, 0xFF)])
def test_bad_scales_of_experts_with_few_rows(B, rows, fmt, byte):
    """In each block of a row, the first, the last and one within: its column is NaN, no other."""
    g = torch.Generator(device="cuda").manual_seed(byte)
    K, N = 512, 40
    w = weights(g, 9, N, K, fmt)
    x = torch.randn((rows, K), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([4] * rows, dtype=torch.int32, device="cuda")
    clean = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2])
    blocks = w[1].shape[-1]
    cols = {0: 0, 7: blocks - 1, 13: blocks // 2, 22: 5, 39: 10}
    for n, b in cols.items():
        w[1][4, n, b] = byte
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = B.fp4_matvec(x, w[0], w[1], fmt, row_expert=ids, weight_scale_2=w[2], workspace=ws)
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[list(cols)] = True
    assert bool(got[:, bad].isnan().all()) and torch.equal(got[:, ~bad], clean[:, ~bad])
    assert B.read_status(ws) == B.MOE_ERR_DATA


@pytest.mark.parametrize("fmt", [0, 1], ids=["mx", "nv"])
@pytest.mark.parametrize("E", [8, 40])
def test_layer_of_tokens_that_name_an_expert_twice(B, E, fmt):
    """The same expert for both slots of a token, for several tokens, and apart."""
    g = torch.Generator(device="cuda").manual_seed(E)
    H, I, k = 512, 288, 3
    w13, w2 = weights(g, E, 2 * I, H, fmt, 114, 122), weights(g, E, H, I, fmt, 114, 122)
    ids = torch.tensor([[3, 3, 3], [3, 5, 5], [7, 0, 3], [1, 2, 1]], dtype=torch.int32, device="cuda")
    x = torch.randn((4, H), generator=g, device="cuda").bfloat16()
    x[3] = x[0]
    w = torch.randn((4, k), generator=g, device="cuda")
    h, y2 = torch.empty((4 * k, I), device="cuda").bfloat16(), torch.empty((4 * k, H), device="cuda")
    out = B.layer_decode(x, ids, w, w13, w2, fmt, h=h, y2=y2)
    flat = ids.view(-1).tolist()
    check(y2, h, w2, flat, 1, fmt)
    same = B.fp4_matvec_swiglu(x, w13[0], w13[1], fmt, row_expert=ids.view(-1), index_div=k, weight_scale_2=w13[2])
    assert torch.equal(same, h) and torch.equal(h[0], h[1]) and torch.equal(h[4], h[5]) and torch.equal(y2[0], y2[2])
    terms = w.double().view(4, k, 1) * y2.double().view(4, k, H)
    # k products and sums in f32, each off by half a step of what has been summed so far
    assert bool(((out.double() - terms.sum(1)).abs() <= k * 2.0 ** -24 * terms.abs().sum(1) + 1e-30).all())


def test_two_streams_at_once(B):
    g = torch.Generator(device="cuda").manual_seed(13)
    w = weights(g, 16, 512, 1024, 0)
    x = torch.randn((2, 8, 1024), generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, 16, (2, 8), generator=g, device="cuda", dtype=torch.int32)
    want = [B.fp4_matvec(x[i], w[0], w[1], 0, row_expert=ids[i]) for i in range(2)]
    out = [[torch.empty_like(want[0]) for _ in range(10)] for _ in range(2)]
    ws = [B.make_workspace(0, 1, 1) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for j in range(10):
        for i in range(2):
            B.fp4_matvec(x[i], w[0], w[1], 0, row_expert=ids[i], out=out[i][j], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i in range(2) for t in out[i])


def test_inputs_that_a_kernel_ahead_still_writes(B):
    """x and the ids of a call are whatever the stream's work ahead of it leaves."""
    g = torch.Generator(device="cuda").manual_seed(14)
    E, H, I, k = 8, 512, 256, 2
    w13, w2 = weights(g, E, 2 * I, H, 0, 116, 122), weights(g, E, H, I, 0, 116, 122)
    xs = torch.randn((20, 3, H), generator=g, device="cuda").bfloat16()
    idss = torch.rand((20, 3, E), generator=g, device="cuda").topk(k, dim=2).indices.to(torch.int32)
    tw = torch.rand((3, k), generator=g, device="cuda")
    want = []
    for x, ids in zip(xs, idss):
        want.append(B.layer_decode(x.contiguous(), ids.contiguous(), tw, w13, w2, 0))
        torch.cuda.synchronize()
    x, ids = torch.empty_like(xs[0]), torch.empty_like(idss[0])
    h, y2, got = torch.empty((6, I), device="cuda").bfloat16(), torch.empty((6, H), device="cuda"), []
    for a, b in zip(xs, idss):
        x.copy_(a)
        ids.copy_(b)
        got.append(B.layer_decode(x, ids, tw, w13, w2, 0, h=h, y2=y2))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
