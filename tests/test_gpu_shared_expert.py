"""A layer of routed 4-bit experts and a dense shared expert, as a model runs it: decode steps
in a captured graph, and a training step of the router and the shared expert with clipped
gradients."""
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


def layer(g, E, H, I, S):
    def weights4(N, K):
        return (torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                torch.randint(116, 121, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8), None)

    mk = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5)  # noqa: E731
    return dict(router=mk(E, H), w13=weights4(2 * I, H), w2=weights4(H, I), s13=mk(2 * S, H).bfloat16(),
                s2=mk(H, S).bfloat16())


@pytest.mark.parametrize("T", [1, 3, 8])
def test_decode(B, T):
    """Routed and shared output of a step, replayed over new tokens, against the sorted layer and
    the plain block: both sides round h to bf16, so that an h on a border may differ by a step
    of 2^-8, and outputs by 2^-8 of their norm at most."""
    E, H, I, S, k = 16, 512, 256, 384, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    p = layer(g, E, H, I, S)
    x = torch.empty((T, H), device="cuda").bfloat16()
    logits = torch.empty((T, E), device="cuda")
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    routed, shared = torch.empty((T, H), device="cuda"), torch.empty((T, H), device="cuda")
    h, y2, sh = (torch.empty((T * k, I), device="cuda").bfloat16(), torch.empty((T * k, H), device="cuda"),
                 torch.empty((T, S), device="cuda").bfloat16())
    ws = B.make_workspace(0, 1, 1)

    def step():
        B.topk_gate(logits, k, out=(ids, w))
        B.layer_decode(x, ids, w, p["w13"], p["w2"], B.MOE_FP4_MX, h=h, y2=y2, out=routed, workspace=ws)
        B.ffn_forward(x, p["s13"], p["s2"], h=sh, out=shared, workspace=ws)

    x.normal_(generator=g)
    logits.copy_(x.float() @ p["router"].T)
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    buffers = B.LayerBuffers(T, k, E, H, I)
    for _ in range(4):
        x.normal_(generator=g)
        logits.copy_(x.float() @ p["router"].T)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = B.layer_forward(x, ids, w, *p["w13"][:2], *p["w2"][:2], buffers).double()
        gate, up = (x.double() @ p["s13"].double().T).split(S, dim=1)
        dense = (torch.nn.functional.silu(gate) * up) @ p["s2"].double().T
        assert float((routed.double() - want).norm() / want.norm()) < 2.0 ** -8
        assert float((shared.double() - dense).norm() / dense.norm()) < 2.0 ** -8
    assert B.read_status(ws) == B.MOE_OK


@pytest.mark.parametrize("T", [96, 300])
def test_training_step(B, T):
    """Gradients of router and shared expert from one loss, clipped together, against autograd
    in 64 bits on the same expert outputs: the shared expert's gradients carry three roundings
    to bf16 (2^-7 of the norm covers them), the router's are f32."""
    E, H, I, S, k = 12, 256, 128, 192, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    p = layer(g, E, H, I, S)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    target = torch.randn((T, H), generator=g, device="cuda")
    logits = x.float() @ p["router"].T
    ids, w = B.topk_gate(logits, k, renorm=True)
    b = B.LayerBuffersFp4(T, k, E, H, I, B.MOE_FP4_MX)
    routed = B.layer_forward_fp4(x, ids, w, p["w13"], p["w2"], b)
    h, gu = torch.empty((T, S), device="cuda").bfloat16(), torch.empty((T, 2 * S), device="cuda").bfloat16()
    shared = B.ffn_forward(x, p["s13"], p["s2"], h=h, gu=gu, out_dtype=torch.float32, workspace=b.workspace)
    dout = 2 * (routed + shared - target)
    _, dw = B.combine_backward(dout, b.y2, b.slot_to_row, w)
    d_router = B.topk_gate_backward(logits, ids, dw, renorm=True).T @ x.float()
    dx, d13, d2 = B.ffn_backward(dout.bfloat16(), x, p["s13"], p["s2"], h, gu, workspace=b.workspace)
    grads = [d_router, d13, d2]
    before = [t.clone() for t in grads]
    norm = float(B.grad_norm(grads))
    assert abs(float(B.clip_grads(grads, 0.5 * norm)) - norm) <= 2.0 ** -24 * norm
    assert B.read_status(b.workspace) == B.MOE_OK

    y = b.y2.double()[b.slot_to_row.long()].view(T, k, H)
    leaves = [t.double().requires_grad_() for t in (p["router"], p["s13"], p["s2"])]
    weights = torch.softmax((x.double() @ leaves[0].T).gather(1, ids.long()), dim=1)
    gate, up = (x.double() @ leaves[1].T).split(S, dim=1)
    out = (weights[:, :, None] * y).sum(1) + (torch.nn.functional.silu(gate) * up) @ leaves[2].T
    (out - target.double()).square().sum().backward()
    want = [leaf.grad for leaf in leaves]
    full = math.sqrt(sum(float(t.square().sum()) for t in want))
    assert abs(norm - full) <= 2.0 ** -7 * full
    for got, t, raw in zip(grads, want, before):
        assert float((raw.double() - t).norm() / t.norm()) < 2.0 ** -7
        scaled = raw.double() * (0.5 * norm / (norm + 1e-6))
        # one rounding to the type, and the norm's and scale's own few 2^-24
        assert float((got.double() - scaled).norm() / scaled.norm()) <= torch.finfo(got.dtype).eps / 2 + 2.0 ** -21
