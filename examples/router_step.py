"""One fine-tuning step of a router over frozen 4-bit experts.

    python examples/router_step.py [--format mx|nv] [--tokens 512] [--steps 4]

Forward, all in the library's kernels: router logits -> moe_topk_gate -> route sort,
4-bit quantisation of the gathered activations, both expert products in 4 bits and
the weighted combine (moe_layer_forward_fp4).  Backward: the loss's gradient at the
layer's output -> moe_combine_backward (gradient of the routing weights, and of the
experts' outputs for experts that train) -> moe_topk_gate_backward -> the router's
weight gradient, and the gradient of x through the routing (moe_gather_backward) when
the experts hand one back.  Weights are random; the loss pulls the layer's output
towards a fixed random target, so it falls from step to step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp4_weight_grouped_gb300 import binding as B  # noqa: E402


class Experts:
    """Frozen 4-bit experts: w13 [E, 2I, H] and w2 [E, H, I]."""

    def __init__(self, E, hidden, inter, fmt, generator):
        def weights(N, K):
            codes = torch.randint(0, 256, (E, N, K // 2), generator=generator, device="cuda", dtype=torch.uint8)
            if fmt == B.MOE_FP4_MX:
                scales = torch.randint(114, 121, (E, N, K // 32), generator=generator, device="cuda", dtype=torch.uint8)
                return codes, scales, None
            scales = torch.randint(0x28, 0x41, (E, N, K // 16), generator=generator, device="cuda", dtype=torch.uint8)
            return codes, scales, torch.full((E,), 2.0 ** -8, device="cuda")

        self.E, self.hidden, self.inter, self.fmt = E, hidden, inter, fmt
        self.w13, self.w2 = weights(2 * inter, hidden), weights(hidden, inter)


class RouterStep:
    """The buffers of a step are made once and used again."""

    def __init__(self, experts, tokens, top_k, renorm=True):
        e = experts
        self.experts, self.k, self.renorm = e, top_k, renorm
        self.buffers = B.LayerBuffersFp4(tokens, top_k, e.E, e.hidden, e.inter, e.fmt)
        nv = e.fmt == B.MOE_FP4_NV
        # Tensor scales a calibration run would give: the largest magnitude / (448 * 6).
        self.x_scale = torch.full((1,), 6.0 / (448 * 6), device="cuda") if nv else None
        self.h_scale = torch.full((1,), 64.0 / (448 * 6), device="cuda") if nv else None

    def forward(self, x, router):
        """x bf16 [T, H], router f32 [E, H] -> out f32 [T, H]."""
        self.x = x
        self.logits = x.float() @ router.T
        self.ids, self.w = B.topk_gate(self.logits, self.k, renorm=self.renorm)
        return B.layer_forward_fp4(x, self.ids, self.w, self.experts.w13, self.experts.w2, self.buffers,
                                   x_scale_2=self.x_scale, h_scale_2=self.h_scale)

    def backward(self, dout):
        """dout f32 [T, H] -> gradient of the router, and dy [T*k, H] (sorted rows), the
        gradient at the experts' outputs."""
        b = self.buffers
        dy, dw = B.combine_backward(dout, b.y2, b.slot_to_row, self.w, dy_dtype=torch.bfloat16)
        dlogits = B.topk_gate_backward(self.logits, self.ids, dw, renorm=self.renorm)
        return dlogits.T @ self.x.float(), dy

    def input_gradient(self, dx_sorted):
        """Gradient at the experts' inputs (sorted rows, from experts that give one) -> at x."""
        return B.gather_backward(dx_sorted, self.buffers.slot_to_row, self.k)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--format", choices=("mx", "nv"), default="mx")
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inter", type=int, default=256)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)
    fmt = B.MOE_FP4_MX if a.format == "mx" else B.MOE_FP4_NV
    experts = Experts(a.experts, a.hidden, a.inter, fmt, g)
    step = RouterStep(experts, a.tokens, a.top_k)
    x = torch.randn((a.tokens, a.hidden), generator=g, device="cuda").to(torch.bfloat16)
    router = torch.randn((a.experts, a.hidden), generator=g, device="cuda") * a.hidden ** -0.5
    target = torch.randn((a.tokens, a.hidden), generator=g, device="cuda")
    losses = []
    for i in range(a.steps):
        out = step.forward(x, router)
        scale = target.norm() / out.norm() if i == 0 else scale
        diff = out * scale - target
        losses.append(float(diff.square().mean()))
        grad, _ = step.backward(2 * scale / diff.numel() * diff)
        router -= 0.05 * grad / grad.norm() * router.norm()
        print(f"step {i}: loss {losses[-1]:.6f}")
    status = B.read_status(step.buffers.workspace)
    if status != B.MOE_OK:
        raise B.MoeError(status, "router step")
    return losses


if __name__ == "__main__":
    main()
