"""Device times of the W4A4 products and of the whole layer at routings that spread tokens over
the experts, and at bands of one length.

    python perf/routed_bands.py [routings] [bands] [k2880] [slope] [layer]     (default: all)

Each figure is the median of several replays of a CUDA graph of calls one after another, so
without the host.  Calls follow one another without a flush of L2: weights of hundreds of MB pass
through it, those of few experts partly stay there, as they do in use.
"share" is of the bytes that the call has to move (touched experts' weights, rows in and out)
at the copy rate of MEASURED_PEAKS.json.
"""
import json
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "perf")]

import operators as ops  # noqa: E402
from fp4_weight_grouped_gb300 import binding as B  # noqa: E402
from fp4_weight_grouped_gb300 import build_lib  # noqa: E402

with open(os.path.join(ROOT, "MEASURED_PEAKS.json")) as f:
    HBM = json.load(f)["hbm_gbs"] * 1e9
FORMATS = (("mx", B.MOE_FP4_MX), ("nv", B.MOE_FP4_NV))
E, TOP_K, HIDDEN, INTER = 256, 6, 4096, 2048


def timed(fn, calls=4, replays=7):
    """Microseconds a call."""
    torch.cuda.synchronize()                  # the side stream reads what the default stream made
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            fn()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(calls):
                fn()
    graph.replay()
    torch.cuda.synchronize()
    took = []
    for _ in range(replays):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b) / calls * 1e3)
    return sorted(took)[replays // 2]


def route(T, k, experts, zipf, gen):
    """k distinct experts a token by the largest of perturbed log-popularities: uniform, or
    Zipf(1.1) with a thirteenth of the experts unused."""
    u = torch.rand((T, experts), generator=gen, device="cuda").clamp_(1e-12, 1 - 1e-7)
    key = -torch.log(-torch.log(u))
    if zipf:
        rank = torch.randperm(experts, generator=gen, device="cuda") + 1
        key += torch.where(rank > experts - experts // 13, -1e9, -1.1 * torch.log(rank.float()))
    return torch.topk(key, k, dim=1).indices.to(torch.int32)


class Products:
    """One call's operands over bands `sizes`, and its two forms."""

    def __init__(self, sizes, K, N, fmt_name, fmt, gen):
        self.sizes, self.K, self.N, self.fmt = sizes, K, N, fmt
        self.rows, self.block = int(sizes.sum()), ops.BLOCK[fmt_name]
        self.touched = int((sizes > 0).sum())
        nv = fmt == B.MOE_FP4_NV
        ac, asc, a2 = ops._act4(self.rows, K, fmt_name, gen)
        wc, wsc, w2 = ops._weights4(sizes.numel(), N, K, fmt_name, gen)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        self.args = (ac, asc, wc, wsc, sizes, fmt)
        self.kw = dict(act_scale_2=a2 if nv else None, weight_scale_2=w2 if nv else None, workspace=self.ws)
        self.h2 = torch.full((1,), 0.006, device="cuda") if nv else None

    def bytes(self, out_row):
        per = self.K // 2 + self.K // self.block
        return self.touched * self.N * per + self.rows * (per + out_row)

    def report(self, what, us, out_row):
        if B.read_status(self.ws) != B.MOE_OK:
            raise SystemExit(f"{what}: status {B.read_status(self.ws)}")
        flops = 2.0 * self.rows * self.K * self.N
        print(f"{what:52s} {us:9.2f} us  share {self.bytes(out_row) / us * 1e6 / HBM * 100:5.1f}%  "
              f"{flops / us / 1e6:8.1f} TFLOP/s", flush=True)

    def plain(self, what, dtype=torch.float32):
        out = torch.empty((self.rows, self.N), dtype=dtype, device="cuda")
        us = timed(lambda: B.fp4_grouped_gemm(*self.args, out=out, **self.kw))
        self.report(f"{what} {'bf16' if dtype == torch.bfloat16 else 'f32'}", us, self.N * out.element_size())

    def swiglu(self, what):
        I = self.N // 2
        out = (torch.empty((self.rows, I // 2), dtype=torch.uint8, device="cuda"),
               torch.empty((self.rows, I // self.block), dtype=torch.uint8, device="cuda"))
        us = timed(lambda: B.fp4_grouped_gemm_swiglu(*self.args, h_scale_2=self.h2, out=out, **self.kw))
        self.report(f"{what} SwiGLU", us, I // 2 + I // self.block)


def generator():
    return torch.Generator(device="cuda").manual_seed(1)


def even(bands, rows):
    return torch.full((bands,), rows, dtype=torch.int32, device="cuda")


def routings():
    for name, T, zipf in (("decode_T64", 64, False), ("decode_T256", 256, False), ("prefill_T4096 Zipf", 4096, True),
                          ("layer_T2048", 2048, False), ("layer_T8192", 8192, False)):
        for f, fmt in FORMATS:
            gen = generator()
            ids = route(T, TOP_K, E, zipf, gen)
            sizes = torch.bincount(ids.flatten().long(), minlength=E).to(torch.int32)
            label = f"{name} ({int((sizes > 0).sum())} of {E} experts)"
            Products(sizes, HIDDEN, 2 * INTER, f, fmt, gen).swiglu(f"{label} {f} w13")
            Products(sizes, INTER, HIDDEN, f, fmt, gen).plain(f"{label} {f} w2")


def bands():
    for rows in (64, 128, 192, 256, 512, 2048):
        for f, fmt in FORMATS:
            Products(even(24, rows), HIDDEN, 2 * INTER, f, fmt, generator()).swiglu(f"24 bands of {rows} {f} w13")
            Products(even(24, rows), INTER, HIDDEN, f, fmt, generator()).plain(f"24 bands of {rows} {f} w2")


def k2880():
    for n, rows in ((6, 4096), (24, 16), (200, 2)):
        for f, fmt in FORMATS:
            for K in (2560, 2880):
                p = Products(even(n, rows), K, 3840, f, fmt, generator())
                p.plain(f"{n} bands of {rows} {f} K {K}")
                p.swiglu(f"{n} bands of {rows} {f} K {K}")


def slope():
    for f, fmt in FORMATS:
        for K in (512, 2048, 4096, 8192):
            p = Products(even(6, 4096), K, 3840, f, fmt, generator())
            for dtype in (torch.bfloat16, torch.float32):
                p.plain(f"6 bands of 4096 {f} K {K}", dtype)
            p.swiglu(f"6 bands of 4096 {f} K {K}")


def layer():
    for f, fmt in FORMATS:
        gen = generator()
        w13, w2 = ops._weights4(E, 2 * INTER, HIDDEN, f, gen), ops._weights4(E, HIDDEN, INTER, f, gen)
        x2, h2 = torch.full((1,), 0.004, device="cuda"), torch.full((1,), 0.01, device="cuda")
        for T in (1, 64, 256, 1024, 8192):
            x = torch.randn((T, HIDDEN), generator=gen, device="cuda").to(torch.bfloat16)
            ids, w = route(T, TOP_K, E, False, gen), torch.rand((T, TOP_K), generator=gen, device="cuda")
            buf = B.LayerBuffersFp4(T, TOP_K, E, HIDDEN, INTER, fmt)
            us = timed(lambda: B.layer_forward_fp4(x, ids, w, w13, w2, buf, x_scale_2=x2, h_scale_2=h2))
            print(f"layer of {T} tokens {f:24s} {us:9.2f} us", flush=True)


if __name__ == "__main__":
    build_lib.build()
    parts = dict(routings=routings, bands=bands, k2880=k2880, slope=slope, layer=layer)
    for name in sys.argv[1:] or parts:
        parts[name]()
        torch.cuda.empty_cache()
