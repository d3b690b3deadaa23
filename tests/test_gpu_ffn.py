"""The dense gated block and its gradient against the formulas in 64 bits.

Products of bf16 are exact in f32 and a sum of K of them in f32 is off by less than 1e-5 of
sum|a b| (K up to 16,384).  What is rounded to bf16 on the way (h, gu, dgu: 2^-8 of each
value at most half a step) is taken from the call's own buffers where the next product is
checked, so each product is held to its own bound, and the stored values to theirs."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8                   # half a step of bf16, relative to the value


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


def inputs(T, H, I, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T + H + I)
    mk = lambda *s, std: (torch.randn(s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    return mk(T, H, std=1.0), mk(2 * I, H, std=H ** -0.5), mk(H, I, std=I ** -0.5), mk(T, H, std=1.0)


def product(got, a, b, what):
    """got = a b^T in f32, perhaps rounded to bf16."""
    a, b = a.double(), b.double()
    want, mass = a @ b.T, a.abs() @ b.abs().T
    tol = 1e-5 * mass + (HALF * want.abs() if got.dtype == torch.bfloat16 else 0) + 1e-30
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), bad.shape)
    return want, 1e-5 * mass


def gate(g, u):
    return g * torch.sigmoid(g) * u


# T, hidden, inter: one token to many, sizes off every tile and stage, one column group.
SHAPES = [(1, 8, 8), (2, 64, 24), (7, 712, 1056), (8, 4096, 128), (9, 264, 136), (33, 72, 520), (64, 4096, 2048),
          (128, 128, 128), (129, 136, 8), (250, 1032, 520), (256, 256, 256), (301, 712, 1056), (513, 520, 264),
          (1024, 64, 1024), (2500, 512, 96),
          # a last round of few items, which are cut in two: outputs, gate, gradients
          (2048, 2560, 64), (2048, 64, 1280), (64, 2560, 1024)]


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("train", [False, True])
def test_forward(B, T, H, I, train):
    x, w13, w2, _ = inputs(T, H, I)
    h = torch.empty((T, I), device="cuda").bfloat16()
    gu = torch.full((T, 2 * I), math.nan, device="cuda").bfloat16() if train else None
    ws = B.make_workspace(0, 1, 1)
    out = B.ffn_forward(x, w13, w2, h=h, gu=gu, workspace=ws, out_dtype=torch.float32)
    assert B.read_status(ws) == B.MOE_OK
    y = x.double() @ w13.double().T
    t = 1e-5 * (x.double().abs() @ w13.double().abs().T)
    if train:
        product(gu, x, w13, "gu")
    g, u, tg, tu = y[:, :I], y[:, I:], t[:, :I], t[:, I:]
    # silu's slope stays below 1.1
    tol = 1.1 * tg * (u.abs() + tu) + (g * torch.sigmoid(g)).abs() * tu + 2 * HALF * gate(g, u).abs() + 1e-30
    assert bool(((h.double() - gate(g, u)).abs() <= tol).all())
    product(out, h, w2, "out")
    low = B.ffn_forward(x, w13, w2, gu=gu, workspace=ws)
    assert torch.equal(low, out.bfloat16())


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("dw", [torch.bfloat16, torch.float32])
def test_backward(B, T, H, I, dw):
    x, w13, w2, dout = inputs(T, H, I)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, gu, dgu = torch.empty((T, I), **bf), torch.empty((T, 2 * I), **bf), torch.empty((T, 2 * I), **bf)
    ws = B.make_workspace(0, 1, 1)
    B.ffn_forward(x, w13, w2, h=h, gu=gu, workspace=ws)
    dx, dw13, dw2 = B.ffn_backward(dout, x, w13, w2, h, gu, dgu=dgu, dw_dtype=dw, workspace=ws)
    assert B.read_status(ws) == B.MOE_OK
    dh, t = dout.double() @ w2.double(), 1e-5 * (dout.double().abs() @ w2.double().abs())
    g, u = gu.double().split(I, dim=1)
    s = torch.sigmoid(g)
    # s (1 + g (1 - s)) passes 0 near g = -1.28: its f32 error is 2^-21 of its terms, not of itself.
    for got, factor, terms in ((dgu[:, :I], u * s * (1 + g * (1 - s)), u.abs()), (dgu[:, I:], g * s, 0)):
        want = dh * factor
        tol = t * factor.abs() + (HALF + 2.0 ** -18) * want.abs() + dh.abs() * terms * 2.0 ** -20 + 1e-30
        assert bool(((got.double() - want).abs() <= tol).all())
    product(dx, dgu, w13.T, "dx")
    product(dw13, dgu.T, x.T, "dw13")
    product(dw2, dout.T, h.T, "dw2")
    # each alone is the same, bit for bit
    for i, whole in enumerate((dx, dw13, dw2)):
        one = [None, None, None]
        one[i] = torch.empty_like(whole)
        B.ffn_backward(dout, x, w13, w2, h, gu, out=one, workspace=ws)
        assert torch.equal(one[i], whole)


@pytest.mark.parametrize("T,H,I", [(4096, 264, 136), (8179, 600, 192), (700, 4104, 2056), (108, 2760, 1832), (1, 1928, 1808)])
def test_long_items_beside_short_ones(B, T, H, I):
    """Launches whose two products have items of very different lengths: few long ones, which go
    first, and the others beside them, with and without a rest that goes round all pairs."""
    test_backward(B, T, H, I, torch.bfloat16)


def test_gradient_is_the_functions(B):
    """Autograd in 64 bits through the whole block: 2^-8 a rounding, three of them in a row
    (gu, dgu, the result), on independent elements: 2^-7 of the norm covers them."""
    x, w13, w2, dout = inputs(200, 256, 192)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, gu = torch.empty((200, 192), **bf), torch.empty((200, 384), **bf)
    B.ffn_forward(x, w13, w2, h=h, gu=gu)
    got = B.ffn_backward(dout, x, w13, w2, h, gu)
    leaves = [t.double().requires_grad_() for t in (x, w13, w2)]
    g, u = (leaves[0] @ leaves[1].T).split(192, dim=1)
    (gate(g, u) @ leaves[2].T).backward(dout.double())
    for a, leaf in zip(got, leaves):
        assert float((a.double() - leaf.grad).norm() / leaf.grad.norm()) < 2.0 ** -7


def test_gradient_is_the_difference(B):
    """A central difference of sum(out * dout) along random directions, in 64 bits."""
    x, w13, w2, dout = inputs(40, 64, 48)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, gu = torch.empty((40, 48), **bf), torch.empty((40, 96), **bf)
    B.ffn_forward(x, w13, w2, h=h, gu=gu)
    grads = B.ffn_backward(dout, x, w13, w2, h, gu, dw_dtype=torch.float32)

    def loss(x, w13, w2):
        g, u = (x @ w13.T).split(48, dim=1)
        return float((gate(g, u) @ w2.T * dout.double()).sum())

    base = [t.double() for t in (x, w13, w2)]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i in range(3):
        d = torch.randn(base[i].shape, generator=gen, device="cuda").double() * float(base[i].abs().mean())
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - 1e-5 * d, base[i] + 1e-5 * d
        want = (loss(*hi) - loss(*lo)) / 2e-5
        got = float((grads[i].double() * d).sum())
        # errors of independent sign: 2^-7 of the root sum of squares, five times over
        assert abs(got - want) <= 5 * 2.0 ** -7 * float((grads[i].double() * d).norm())


@pytest.mark.parametrize("T", [3, 70, 300])
def test_strided_x_and_rows_behind(B, T):
    """Rows of x apart from one another, and nothing written behind the last row."""
    H, I = 264, 72
    x, w13, w2, dout = inputs(T, H, I)
    wide = torch.full((T, H + 24), math.nan, device="cuda").bfloat16()
    wide[:, 8:8 + H] = x
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, gu, out = (torch.full((T + 3, n), 7.0, **bf) for n in (I, 2 * I, H))
    B.ffn_forward(wide[:, 8:8 + H], w13, w2, h=h[:T], gu=gu[:T], out=out[:T])
    assert torch.equal(out[:T], B.ffn_forward(x, w13, w2, gu=torch.empty_like(gu[:T])))
    dgu, dx = torch.full((T + 3, 2 * I), 7.0, **bf), torch.full((T + 3, H), 7.0, **bf)
    dw13, dw2 = torch.full((2 * I + 1, H), 7.0, **bf), torch.full((H + 1, I), 7.0, **bf)
    B.ffn_backward(dout, wide[:, 8:8 + H], w13, w2, h[:T], gu[:T], dgu=dgu[:T], out=(dx[:T], dw13[:2 * I], dw2[:H]))
    want = B.ffn_backward(dout, x, w13, w2, h[:T], gu[:T])
    assert torch.equal(dx[:T], want[0]) and torch.equal(dw13[:2 * I], want[1]) and torch.equal(dw2[:H], want[2])
    for t in (h[T:], gu[T:], out[T:], dgu[T:], dx[T:], dw13[2 * I:], dw2[H:]):
        assert bool((t == 7).all())
    few = torch.full((T + 3, H), 7.0, **bf)
    B.ffn_forward(wide[:, 8:8 + H], w13, w2, out=few[:T])
    assert bool((few[T:] == 7).all()) and torch.equal(few[:T], B.ffn_forward(x, w13, w2))


def test_no_tokens(B):
    x, w13, w2, dout = inputs(4, 64, 32)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, gu = torch.empty((0, 32), **bf), torch.empty((0, 64), **bf)
    assert B.ffn_forward(x[:0], w13, w2, h=h, gu=gu).shape == (0, 64)
    for dw in (torch.bfloat16, torch.float32):
        out = (torch.empty((0, 64), **bf), torch.full((64, 64), 7.0, device="cuda", dtype=dw),
               torch.full((64, 32), 7.0, device="cuda", dtype=dw))
        B.ffn_backward(dout[:0], x[:0], w13, w2, h, gu, out=out)
        assert bool((out[1] == 0).all()) and bool((out[2] == 0).all())


@pytest.mark.parametrize("T", [5, 140])
def test_tokens_that_are_not_finite_stay_theirs(B, T):
    x, w13, w2, _ = inputs(T, 128, 64)
    clean = B.ffn_forward(x, w13, w2)
    x[2, 5], x[4, 7] = math.nan, math.inf
    got = B.ffn_forward(x, w13, w2)
    assert bool(torch.isnan(got[2]).all())
    rest = [i for i in range(T) if i not in (2, 4)]
    assert torch.equal(got[rest], clean[rest])


def test_gates_at_the_ends(B):
    """g of 0, of either sign and far out: no overflow on the way to the gradient."""
    H = I = 64
    g = torch.tensor([0.0, -0.0, 1.0, -1.0, 20.0, -20.0, 88.0, -88.0, 200.0, -200.0, 1e4, -1e4, 1e30, -1e30], device="cuda")
    T = g.numel()
    gu = torch.cat([g[:, None].expand(T, I), torch.full((T, I), 2.0, device="cuda")], dim=1).bfloat16().contiguous()
    w2 = torch.eye(H, device="cuda").bfloat16()
    dout = torch.ones((T, H), device="cuda").bfloat16()
    x, w13 = torch.ones((T, H), device="cuda").bfloat16(), torch.ones((2 * I, H), device="cuda").bfloat16()
    dgu = torch.empty_like(gu)
    B.ffn_backward(dout, x, w13, w2, torch.ones((T, I), device="cuda").bfloat16(), gu, dgu=dgu)
    g64 = gu[:, :I].double()
    s = torch.sigmoid(g64)
    for got, want in ((dgu[:, :I], 2 * s * (1 + g64 * torch.sigmoid(-g64))), (dgu[:, I:], g64 * s)):
        assert bool(((got.double() - want).abs() <= (HALF + 2.0 ** -18) * want.abs() + 2.0 ** -126).all())


def test_graphs_and_streams(B):
    x, w13, w2, dout = inputs(300, 256, 128)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, gu, dgu, out = (torch.empty((300, n), **bf) for n in (128, 256, 256, 256))
    grads = (torch.empty_like(x), torch.empty_like(w13), torch.empty_like(w2))
    ws = B.make_workspace(0, 1, 1)

    def step(stream=None):
        B.ffn_forward(x, w13, w2, h=h, gu=gu, out=out, workspace=ws, stream=stream)
        B.ffn_backward(dout, x, w13, w2, h, gu, dgu=dgu, out=grads, workspace=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    x.mul_(0.5)
    dout.neg_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    first = [t.clone() for t in (out, *grads)]
    step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (out, *grads)))


def test_two_streams_at_once(B):
    args = [inputs(n, 256, 192, seed=n) for n in (130, 260)]
    bf = dict(dtype=torch.bfloat16, device="cuda")

    def step(i, s, b):
        x, w13, w2, dout = args[i]
        B.ffn_forward(x, w13, w2, h=b["h"], gu=b["gu"], out=b["out"], workspace=b["ws"], stream=s)
        B.ffn_backward(dout, x, w13, w2, b["h"], b["gu"], dgu=b["dgu"], out=b["grads"], workspace=b["ws"], stream=s)

    def buffers(i):
        x, w13, w2, _ = args[i]
        T = x.shape[0]
        return dict(h=torch.empty((T, 192), **bf), gu=torch.empty((T, 384), **bf), dgu=torch.empty((T, 384), **bf),
                    out=torch.empty_like(x), grads=tuple(torch.empty_like(t) for t in (x, w13, w2)), ws=B.make_workspace(0, 1, 1))

    want = [buffers(i) for i in range(2)]
    for i in range(2):
        step(i, None, want[i])
    torch.cuda.synchronize()
    many = [[buffers(i) for _ in range(6)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for j in range(6):
        for i in range(2):
            step(i, streams[i], many[i][j])
    torch.cuda.synchronize()
    for i in range(2):
        for b in many[i]:
            assert all(torch.equal(p, q) for p, q in zip((b["out"], *b["grads"]), (want[i]["out"], *want[i]["grads"])))


@pytest.mark.parametrize("T", [4, 200])
def test_inputs_that_a_kernel_ahead_still_writes(B, T):
    """Both products in a chain: the second starts under the first's end, the first waits for
    what is ahead of it."""
    x, w13, w2, _ = inputs(T, 512, 384)
    xs = [x * (0.5 + 0.1 * i) for i in range(12)]
    want = []
    for a in xs:
        want.append(B.ffn_forward(a, w13, w2))
        torch.cuda.synchronize()
    now, h, got = torch.empty_like(x), torch.empty((T, 384), device="cuda").bfloat16(), []
    for a in xs:
        now.copy_(a)
        got.append(B.ffn_forward(now, w13, w2, h=h))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
