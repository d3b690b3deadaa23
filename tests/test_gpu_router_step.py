"""The router fine-tuning example: its gradients against autograd through a plain
64-bit form of the gate and the combine on the same expert outputs, and its loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__ as g
    g.build()
    spec = importlib.util.spec_from_file_location("router_step", os.path.join(ROOT, "examples", "router_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_loss_falls(ex, fmt):
    losses = ex.main(["--format", fmt, "--tokens", "256", "--steps", "5"])
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_is_autograds(ex, renorm):
    """f32 products of the example (logits, router gradient) and f32 gradients of the
    gate and combine against autograd in 64 bits: 1e-4 of the gradient's norm covers K =
    256 to 4,096 additions in f32 several times over."""
    B = ex.B
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, I, E, k = 96, 256, 128, 12, 3
    step = ex.RouterStep(ex.Experts(E, H, I, B.MOE_FP4_MX, g), T, k, renorm)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    router = torch.randn((E, H), generator=g, device="cuda") * H ** -0.5
    dout = torch.randn((T, H), generator=g, device="cuda")
    out = step.forward(x, router)
    grad, dy = step.backward(dout)
    assert B.read_status(step.buffers.workspace) == B.MOE_OK
    y = step.buffers.y2.double().requires_grad_()
    r64 = router.double().requires_grad_()
    logits = x.double() @ r64.T
    top = logits.topk(k, dim=1).indices
    assert torch.equal(top.int(), step.ids)
    p = torch.softmax(logits.gather(1, top) if renorm else logits, dim=1)
    w = p if renorm else p.gather(1, top)
    ref = (w[:, :, None] * y[step.buffers.slot_to_row.long()].view(T, k, H)).sum(1)
    ref.backward(dout.double())
    assert float((out.double() - ref.detach()).norm() / ref.detach().norm()) < 1e-5
    assert float((grad.double() - r64.grad).norm() / r64.grad.norm()) < 1e-4
    assert float((dy.double() - y.grad).norm() / y.grad.norm()) < 2.0 ** -8      # dy is bf16
    dx = step.input_gradient(y.grad.float())
    want = y.grad[step.buffers.slot_to_row.long()].view(T, k, H).sum(1)
    assert float((dx.double() - want).norm() / want.norm()) < 1e-6
