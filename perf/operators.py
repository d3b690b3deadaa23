"""Workloads of the 4-bit and gradient operators of the routed-expert layer.

Each case is one pass through one operator at sizes the layer meets: router gate
(forward and gradient), quantisation to MXFP4 / NVFP4, grouped products of 4-bit
activations with 4-bit expert weights, and the gradient of the weighted unsort
and of the sort.  With ``own`` false, run() computes the plain form in float32
from elementary torch operations; with ``own`` true it calls the library.
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # Router of one decode step: 64 tokens over 256 experts; latency counts.
        dict(name="gate_decode", op="gate", T=64, E=256, k=6, renorm=False, dtype="f32"),
        # Router of a long prefill or training step, renormalised weights.
        dict(name="gate_layer", op="gate", T=8192, E=256, k=6, renorm=True, dtype="bf16"),
        # Sorted activations of one decode step (384 rows of 4096) to MXFP4.
        dict(name="quant_decode", op="quant", T=64, E=256, k=6, K=4096, fmt="mx", dtype="bf16"),
        # Sorted activations of the full layer (49152 rows) to MXFP4.
        dict(name="quant_layer", op="quant", T=8192, E=256, k=6, K=4096, fmt="mx", dtype="bf16"),
        # f32 hidden rows (k = 1: no choices to gather) to NVFP4, 3001 ragged rows.
        dict(name="quant_nv_f32", op="quant", T=3001, E=16, k=1, K=2080, fmt="nv", dtype="f32"),
        # w13 product of a decode step: 1 or 2 rows an expert, weights streamed once.
        dict(name="gemm_decode_w13", op="gemm", T=64, E=256, k=6, K=4096, N=4096, fmt="mx", out="f32", zipf=False),
        # w2 product of a prefill with Zipf popularity: bands from 0 to thousands of rows.
        dict(name="gemm_prefill_w2", op="gemm", T=4096, E=256, k=6, K=2048, N=4096, fmt="nv", out="bf16", zipf=True),
        # A small model's odd sizes: K off every tile, N off the 128-row tile.
        dict(name="gemm_odd", op="gemm", T=301, E=12, k=2, K=1056, N=712, fmt="mx", out="f32", zipf=False),
        # Both expert products with SwiGLU and requantisation between, full layer.
        dict(name="mlp_layer", op="mlp", T=8192, E=256, k=6, hidden=4096, inter=2048, fmt="mx", zipf=False),
        # The same pair for a decode step of 256 tokens in NVFP4.
        dict(name="mlp_decode", op="mlp", T=256, E=256, k=6, hidden=4096, inter=2048, fmt="nv", zipf=False),
        # Gradients of unsort and sort in a small fine-tuning step, ragged columns.
        dict(name="unsort_grad_small", op="grad", T=250, E=64, k=6, N=1028, dtype="bf16"),
        # The same for the full layer.
        dict(name="unsort_grad_layer", op="grad", T=8192, E=256, k=6, N=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _mult(rng, lo, hi, m):
    v = max(lo, _log(rng, lo, hi) // m * m)
    return v + m if v == 3072 else v


def draw(rng):
    op = rng.choice(["gate", "quant", "gemm", "mlp", "grad"])
    E = _log(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 8192)
    fmt = rng.choice(["mx", "nv"])
    zipf = rng.random() < 0.5
    if op == "gate":
        return dict(op=op, T=T, E=E, k=k, renorm=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]))
    if op == "quant":
        return dict(op=op, T=T, E=E, k=min(k, 6), K=_mult(rng, 32, 4096, 32), fmt=fmt, dtype=rng.choice(["f32", "bf16"]))
    if op == "gemm":
        return dict(op=op, T=T, E=E, k=min(k, 6), K=_mult(rng, 64, 4096, 32), N=_mult(rng, 8, 4096, 4), fmt=fmt,
                    out=rng.choice(["f32", "bf16"]), zipf=zipf)
    if op == "mlp":
        return dict(op=op, T=T, E=E, k=min(k, 6), hidden=_mult(rng, 64, 4096, 32), inter=_mult(rng, 64, 2048, 32),
                    fmt=fmt, zipf=zipf)
    return dict(op=op, T=T, E=E, k=min(k, 6), N=_mult(rng, 4, 4096, 4), dtype=rng.choice(["f32", "bf16"]))


def _scale_bytes(fmt, K):
    return K // BLOCK[fmt]


def _touched(c):
    """Experts with at least one row, in expectation (uniform choice)."""
    return min(c["E"], c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"]))


def work(c):
    op = c["op"]
    rows = c["T"] * c["k"]
    if op == "gate":
        e = 4 if c["dtype"] == "f32" else 2
        # logits in and their gradient out, ids and weights out, d(weights) in
        return {"bytes": c["T"] * c["E"] * 2 * e + rows * 12, "flops": c["T"] * c["E"] * (10 + c["k"])}
    if op == "quant":
        e = 4 if c["dtype"] == "f32" else 2
        out = c["K"] / 2 + _scale_bytes(c["fmt"], c["K"]) + c["K"] * (2 if c["fmt"] == "mx" else 4)
        return {"bytes": c["T"] * c["K"] * e + rows * (out + 4), "flops": rows * c["K"] * 4}
    if op == "gemm":
        per = c["K"] / 2 + _scale_bytes(c["fmt"], c["K"])
        o = 4 if c["out"] == "f32" else 2
        return {"bytes": (_touched(c) * c["N"] + rows) * per + rows * c["N"] * o, "flops": 2.0 * rows * c["K"] * c["N"]}
    if op == "mlp":
        p1 = c["hidden"] / 2 + _scale_bytes(c["fmt"], c["hidden"])
        p2 = c["inter"] / 2 + _scale_bytes(c["fmt"], c["inter"])
        b = _touched(c) * (2 * c["inter"] * p1 + c["hidden"] * p2) + rows * (p1 + 2 * c["hidden"])
        return {"bytes": b, "flops": 2.0 * rows * 3 * c["hidden"] * c["inter"]}
    e = 4 if c["dtype"] == "f32" else 2
    # dout in, y (f32) in, dy out, w in, dw out; then the sorted gradient in, dx out
    return {"bytes": c["T"] * c["N"] * e + rows * c["N"] * (4 + e) + rows * 12 + rows * c["N"] * e + c["T"] * c["N"] * e,
            "flops": rows * c["N"] * 4}


# ------------------------------------------------------------------- inputs

def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _routing(c, g):
    """k distinct experts a token (uniform, or Zipf(1.1) with a few unused), and
    the stable expert-sorted order of the slots."""
    T, E, k = c["T"], c["E"], c["k"]
    keys = torch.rand((T, E), generator=g, device="cuda").clamp_min_(1e-20)
    keys = -torch.log(-torch.log(keys).clamp_min(1e-20))
    if c.get("zipf"):
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        logp = -1.1 * torch.log(rank.float())
        logp[rank > max(k, E - E // 13)] = -1e9
        keys += logp
    ids = torch.topk(keys, k, dim=1).indices.to(torch.int32)
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    s2r = torch.empty_like(order)
    s2r[order] = torch.arange(order.numel(), device="cuda")
    sizes = torch.bincount(flat, minlength=E)
    return ids, sizes.to(torch.int32), order.to(torch.int32), s2r.to(torch.int32), sizes.tolist()


def _act4(rows, K, fmt, g):
    """Quantised N(0, 1) activations: codes, scales and the NVFP4 tensor scale."""
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, K // BLOCK[fmt]), dtype=torch.uint8, device="cuda")
    ts = torch.full((1,), 6.0 / (448 * 6), device="cuda")
    for r in range(0, rows, 8192):
        x = torch.randn((min(8192, rows - r), K), generator=g, device="cuda")
        codes[r:r + 8192], scales[r:r + 8192], _ = _quantise(x, fmt, ts)
    return codes, scales, ts


def _weights4(E, N, K, fmt, g):
    """Uniform codes; E8M0 exponents -14..-6, or E4M3 scales 0.25..2 under a
    per-expert scale: sums over K of a few thousand come out of order one."""
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "mx":
        scales = torch.randint(113, 122, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    else:
        scales = torch.randint(0x28, 0x41, (E, N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    ws2 = 2.0 ** torch.randint(-9, -5, (E,), generator=g, device="cuda").float()
    ws2 = ws2 * (1 + torch.randint(0, 8, (E,), generator=g, device="cuda").float() / 8)
    return codes, scales, ws2


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, E, k = c["op"], c["T"], c["E"], c["k"]
    rows = T * k
    # The status word a user's program clears once and passes to every call.
    s = dict(case=c, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "gate":
        s["logits"] = (torch.randn((T, E), generator=g, device="cuda") * 1.5).to(_dt(c["dtype"]))
        s["dw"] = torch.randn((T, k), generator=g, device="cuda")
        s["ids"], s["w"] = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
        s["dlogits"] = torch.empty_like(s["logits"])
        return s
    ids, sizes, order, s2r, host = _routing(c, g)
    s |= dict(sizes=sizes, order=order, s2r=s2r, host=host)
    if op == "quant":
        K = c["K"]
        x = torch.randn((T, K), generator=g, device="cuda")
        # a few channels an order of magnitude larger, as trained activations have
        x *= 1 + 9 * (torch.rand((K,), generator=g, device="cuda") < 0.02)
        s["x"] = x.to(_dt(c["dtype"]))
        s["ts"] = torch.full((1,), 60.0 / (448 * 6), device="cuda")
        s["codes"] = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((rows, K // BLOCK[c["fmt"]]), dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty((rows, K), dtype=torch.bfloat16 if c["fmt"] == "mx" else torch.float32, device="cuda")
    elif op == "gemm":
        s["a"] = _act4(rows, c["K"], c["fmt"], g)
        s["w13"] = _weights4(E, c["N"], c["K"], c["fmt"], g)
        s["y"] = torch.empty((rows, c["N"]), dtype=_dt(c["out"]), device="cuda")
    elif op == "mlp":
        H, I = c["hidden"], c["inter"]
        s["a"] = _act4(rows, H, c["fmt"], g)
        s["w13"] = _weights4(E, 2 * I, H, c["fmt"], g)
        s["w2"] = _weights4(E, H, I, c["fmt"], g)
        # Calibrated once from sample data in use; here from the inputs' spread.
        s["hs"] = torch.full((1,), 16.0 * H / 4096 / (448 * 6), device="cuda")
        s["h"] = (torch.empty((rows, I // 2), dtype=torch.uint8, device="cuda"),
                  torch.empty((rows, I // BLOCK[c["fmt"]]), dtype=torch.uint8, device="cuda"))
        s["y"] = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    else:
        N, dt = c["N"], _dt(c["dtype"])
        s["w"] = torch.rand((T, k), generator=g, device="cuda") * 0.3
        s["dout"] = torch.randn((T, N), generator=g, device="cuda").to(dt)
        s["y"] = torch.randn((rows, N), generator=g, device="cuda")
        s["dxs"] = torch.randn((rows, N), generator=g, device="cuda").to(dt)
        s["dy"], s["dw"] = torch.empty((rows, N), dtype=dt, device="cuda"), torch.empty((T, k), device="cuda")
        s["dx"] = torch.empty((T, N), dtype=dt, device="cuda")
    return s


# -------------------------------------------------------------- plain forms

_tables = {}


def _table(name):
    if name not in _tables:
        mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
        e2m1 = torch.cat([mags, -mags]) + 0.0
        b = torch.arange(256, device="cuda")
        _tables["mags"] = mags
        _tables["pairs"] = torch.stack([e2m1[b % 16], e2m1[b // 16]], dim=1)      # low nibble first
        _tables["mx"] = torch.ldexp(torch.ones(256, device="cuda"), (b - 127).float())
        _tables["nv"] = b.to(torch.uint8).view(torch.float8_e4m3fn).float()
    return _tables[name]


def _quantise(x, fmt, ts):
    """float32 rows -> codes, scale bytes, and the values they stand for."""
    R, K = x.shape
    xb = x.view(R, K // BLOCK[fmt], BLOCK[fmt])
    amax = xb.abs().amax(dim=2)
    if fmt == "mx":
        byte = ((amax.view(torch.int32) >> 23) - 2).clamp_min(0)     # floor(log2) - 2, biased
        inv = torch.ldexp(torch.ones_like(amax), (127 - byte).float())
        scale = _table("mx")[byte]
        byte = byte.to(torch.uint8)
    else:
        s8 = (amax / (6 * ts)).clamp_max(448).to(torch.float8_e4m3fn)
        scale = s8.float()
        inv = 1 / (scale * ts)
        inv = torch.where(inv < math.inf, inv, 0)
        byte = s8.view(torch.uint8)
    q = xb * inv[:, :, None]
    m = q.abs()
    # nearest magnitude; a tie goes to the even mantissa
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    neg = (q < 0) & (code > 0)
    mag = _table("mags")[code.int()]
    values = torch.where(neg, -mag, mag) * scale[:, :, None]
    if fmt == "nv":
        values = values * ts
    nib = (code + 8 * neg.to(torch.uint8)).view(R, K // 2, 2)
    return nib[:, :, 0] | (nib[:, :, 1] << 4), byte, values.view(R, K)


def _values(codes, scales, fmt):
    """Codes [R, K/2] and block scales -> float32 [R, K]."""
    R = codes.shape[0]
    v = _table("pairs")[codes.int()].view(R, scales.shape[1], BLOCK[fmt])
    return (v * _table(fmt)[scales.int()][:, :, None]).view(R, -1)


def _bands(s, a, w, fmt, ts, each):
    """One product for each expert that has rows, as each has its own weights."""
    codes, scales, ws2 = w
    r = 0
    for e, n in enumerate(s["host"]):
        if n:
            y = _values(a[0][r:r + n], a[1][r:r + n], fmt) @ _values(codes[e], scales[e], fmt).T
            each(r, r + n, y * (ws2[e] * ts) if fmt == "nv" else y)
            r += n


def _plain(s):
    c = s["case"]
    op, k = c["op"], c["k"]
    if op == "gate":
        l = s["logits"].float()
        ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
        if c["renorm"]:
            l = torch.gather(l, 1, ids)
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
        w = p if c["renorm"] else torch.gather(p, 1, ids)
        dot = (w * s["dw"]).sum(dim=1, keepdim=True)
        if c["renorm"]:
            dl = torch.zeros(s["logits"].shape, device="cuda").scatter(1, ids, w * (s["dw"] - dot))
        else:
            dl = (p * -dot).scatter_add(1, ids, w * s["dw"])
        return {"ids": ids.to(torch.int32), "w": w, "dlogits": dl.to(s["logits"].dtype)}
    if op == "quant":
        x = s["x"][s["order"].long() // k].float()
        return {"values": _quantise(x, c["fmt"], s["ts"])[2].to(s["values"].dtype)}
    if op == "gemm":
        y = torch.empty_like(s["y"])
        _bands(s, s["a"], s["w13"], c["fmt"], s["a"][2], lambda r0, r1, v: y[r0:r1].copy_(v))
        return {"y": y}
    if op == "mlp":
        I = c["inter"]
        hc, hs, y = torch.empty_like(s["h"][0]), torch.empty_like(s["h"][1]), torch.empty_like(s["y"])

        def gate(r0, r1, v):
            g, u = v[:, :I], v[:, I:]
            hc[r0:r1], hs[r0:r1], _ = _quantise(g / (1 + torch.exp(-g)) * u, c["fmt"], s["hs"])

        _bands(s, s["a"], s["w13"], c["fmt"], s["a"][2], gate)
        _bands(s, (hc, hs), s["w2"], c["fmt"], s["hs"], lambda r0, r1, v: y[r0:r1].copy_(v))
        return {"y": y}
    T, N = c["T"], c["N"]
    at = s["s2r"].long()
    dout = s["dout"].float()
    dy = torch.empty((T * k, N), dtype=s["dout"].dtype, device="cuda")
    dy[at] = (s["w"][:, :, None] * dout[:, None, :]).view(T * k, N).to(dy.dtype)
    dw = (s["y"][at].view(T, k, N) * dout[:, None, :]).sum(dim=2)
    dx = s["dxs"][at].float().view(T, k, N).sum(dim=1).to(s["dxs"].dtype)
    return {"dy": dy, "dw": dw, "dx": dx}


# -------------------------------------------------------- the library's calls

def _library(s):
    from fp4_weight_grouped_gb300 import binding as B

    c = s["case"]
    op, k = c["op"], c["k"]
    if op == "gate":
        ids, w = B.topk_gate(s["logits"], k, renorm=c["renorm"], out=(s["ids"], s["w"]))
        dl = B.topk_gate_backward(s["logits"], ids, s["dw"], renorm=c["renorm"], out=s["dlogits"])
        return {"ids": ids, "w": w, "dlogits": dl}
    fmt = B.MOE_FP4_MX if c.get("fmt") == "mx" else B.MOE_FP4_NV
    nv = c.get("fmt") == "nv"
    if op == "quant":
        B.fp4_quantize(s["x"], fmt, row_index=s["order"], index_div=k, tensor_scale=s["ts"] if nv else None,
                       out=(s["codes"], s["scales"]), values=s["values"], workspace=s["ws"])
        return {"values": s["values"]}
    if op == "gemm":
        (ac, asc, ts), (wc, wsc, ws2) = s["a"], s["w13"]
        y = B.fp4_grouped_gemm(ac, asc, wc, wsc, s["sizes"], fmt, act_scale_2=ts if nv else None,
                               weight_scale_2=ws2 if nv else None, out=s["y"], workspace=s["ws"])
        return {"y": y}
    if op == "mlp":
        (ac, asc, ts), (c13, s13, g13), (c2, s2, g2) = s["a"], s["w13"], s["w2"]
        hc, hs = B.fp4_grouped_gemm_swiglu(ac, asc, c13, s13, s["sizes"], fmt, act_scale_2=ts if nv else None,
                                           weight_scale_2=g13 if nv else None, h_scale_2=s["hs"] if nv else None,
                                           out=s["h"], workspace=s["ws"])
        y = B.fp4_grouped_gemm(hc, hs, c2, s2, s["sizes"], fmt, act_scale_2=s["hs"] if nv else None,
                               weight_scale_2=g2 if nv else None, out=s["y"], workspace=s["ws"])
        return {"y": y}
    dy, dw = B.combine_backward(s["dout"], s["y"], s["s2r"], s["w"], out=(s["dy"], s["dw"]))
    dx = B.gather_backward(s["dxs"], s["s2r"], k, out=s["dx"])
    return {"dy": dy, "dw": dw, "dx": dx}


def run(s):
    return _library(s) if own else _plain(s)


# ------------------------------------------------- the definitions in 64 bits

def _x_e2m1(nibbles):
    """e2m1 from its bits: sign, two exponent bits (bias 1), one mantissa bit."""
    sign, e, f = nibbles >> 3 & 1, nibbles >> 1 & 3, (nibbles & 1).double()
    mag = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.pow(2.0, (e - 1).double()))
    return torch.where(sign == 1, -mag, mag)


def _x_scale(b, fmt):
    b = b.long()
    if fmt == "mx":
        return torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), (b - 127).double())
    e, m = b >> 3 & 15, (b & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(b >= 128, -mag, mag)


def _x_values(codes, scales, fmt):
    c = codes.to(torch.int16)
    v = torch.stack([_x_e2m1(c & 15), _x_e2m1(c >> 4)], dim=2).flatten(1)
    return v * _x_scale(scales, fmt).repeat_interleave(BLOCK[fmt], dim=1)


def _x_round(v, fmt, ts):
    """The values nearest to v (float64 rows) in the format; ties to even."""
    v = v.unflatten(1, (-1, BLOCK[fmt]))
    top = v.abs().amax(dim=2, keepdim=True)
    if fmt == "mx":
        unit = torch.pow(2.0, (torch.frexp(top).exponent.double() - 1 - 2).clamp(-127, 125))
    else:
        t = (top / (6 * ts)).clamp_max(448)
        step = torch.pow(2.0, (torch.frexp(t).exponent.double() - 1).clamp_min(-6) - 3)
        unit = torch.round(t / step) * step * ts
    m = torch.where(unit > 0, v.abs() / unit.clamp_min(1e-300), 0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp_max(6)
    return (torch.sign(v) * m * unit).flatten(1)


def exact(c, seed):
    s = prepare(c, seed)
    op, k, T = c["op"], c["k"], c["T"]
    if op == "gate":
        l = s["logits"].double()
        ids = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
        chosen = torch.zeros_like(l, dtype=torch.bool).scatter(1, ids, True)
        if c["renorm"]:
            l = torch.where(chosen, l, -math.inf)
        p = torch.softmax(l, dim=1)
        dp = torch.zeros_like(l).scatter(1, ids, s["dw"].double())
        return {"ids": ids.to(torch.int32), "w": p.gather(1, ids), "dlogits": p * (dp - (p * dp).sum(1, keepdim=True))}
    fmt = c.get("fmt")
    if op == "quant":
        v = torch.empty((T * k, c["K"]), dtype=torch.float64, device="cuda")
        x = _x_round(s["x"].double(), fmt, s["ts"].double())
        return {"values": torch.index_select(x, 0, s["order"].long() // k, out=v)}
    if op in ("gemm", "mlp"):
        n_out = c["N"] if op == "gemm" else c["hidden"]
        y = torch.empty((T * k, n_out), dtype=torch.float64, device="cuda")
        r, I = 0, c.get("inter")
        for e, n in enumerate(s["host"]):
            if n == 0:
                continue
            a = _x_values(s["a"][0][r:r + n], s["a"][1][r:r + n], fmt)
            w = _x_values(s["w13"][0][e], s["w13"][1][e], fmt)
            if fmt == "nv":
                a, w = a * s["a"][2].double(), w * s["w13"][2][e].double()
            v = torch.einsum("rk,nk->rn", a, w)
            if op == "mlp":
                h = _x_round(v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:], fmt, s["hs"].double())
                w = _x_values(s["w2"][0][e], s["w2"][1][e], fmt)
                v = torch.einsum("rk,nk->rn", h, w * s["w2"][2][e].double() if fmt == "nv" else w)
            y[r:r + n] = v
            r += n
        return {"y": y}
    N = c["N"]
    token = s["order"].long() // k
    choice = s["order"].long() % k
    dy = s["w"].double()[token, choice][:, None] * s["dout"].double()[token]
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    dw[token, choice] = torch.einsum("rn,rn->r", s["dout"].double()[token], s["y"].double())
    dx = torch.zeros((T, N), dtype=torch.float64, device="cuda").index_add_(0, token, s["dxs"].double())
    return {"dy": dy, "dw": dw, "dx": dx}
