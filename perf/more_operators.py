"""Workloads of the operators around the routed experts: products of a few tokens with
4-bit weights, the dense gated feed-forward block (the shared expert) and its gradient,
and the global norm and clipping of gradients.

Each case is one pass through one operator.  With ``own`` false, run() computes the plain
form in float32 from elementary torch operations; with ``own`` true it calls the library.
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One token through the routed experts, six of 256: what a chat's next token waits for.
        dict(name="decode_1", op="decode", T=1, E=256, k=6, hidden=4096, inter=2048, fmt="mx"),
        # Eight streams decoding together in NVFP4: nearly every slot has an expert of its own.
        dict(name="decode_8", op="decode", T=8, E=256, k=6, hidden=4096, inter=2048, fmt="nv"),
        # A dense 4-bit projection of four tokens: one weight matrix, read once.
        dict(name="matvec_dense", op="matvec", T=4, E=1, k=1, K=4096, N=4096, fmt="mx", out="bf16"),
        # A small model's odd sizes: rows of scales off every vector width, columns off every tile.
        dict(name="matvec_odd", op="matvec", T=5, E=12, k=2, K=1056, N=713, fmt="nv", out="f32"),
        # The shared expert for one token: its weights once through the chip.
        dict(name="ffn_1", op="ffn", T=1, hidden=4096, inter=2048),
        # The shared expert of a decode batch.
        dict(name="ffn_64", op="ffn", T=64, hidden=4096, inter=2048),
        # A small model's prompt with sizes off every tile.
        dict(name="ffn_odd", op="ffn", T=301, hidden=712, inter=1056),
        # The shared expert over a prefill.
        dict(name="ffn_prefill", op="ffn", T=4096, hidden=4096, inter=2048),
        # A training step of a small block, ragged in every dimension.
        dict(name="train_small", op="train", T=250, hidden=1032, inter=520),
        # A training step of the layer's shared expert: forward, and gradients of x and weights.
        dict(name="train_layer", op="train", T=8192, hidden=4096, inter=2048),
        # Gradients of a small router and block, clipped: a handful of launches' worth of work.
        dict(name="clip_small", op="clip", layers=2, E=32, hidden=513, inter=260, dtype="f32", below=False),
        # Routers, shared experts and norms of 24 layers: 1.4 GB of gradients.
        dict(name="clip_layers", op="clip", layers=24, E=256, hidden=4096, inter=2048, dtype="bf16", below=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _mult(rng, lo, hi, m):
    return max(lo, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["decode", "matvec", "ffn", "train", "clip"])
    fmt = rng.choice(["mx", "nv"])
    if op in ("decode", "matvec"):
        T, E = _log(rng, 1, 16), _log(rng, 1, 256)
        k = min(E, rng.randint(1, 8), 64 // T)
        if op == "decode":
            return dict(op=op, T=T, E=E, k=k, hidden=_mult(rng, 32, 4096, 32), inter=_mult(rng, 32, 2048, 32), fmt=fmt)
        return dict(op=op, T=T, E=E, k=k, K=_mult(rng, 32, 4096, 32), N=_log(rng, 1, 4096), fmt=fmt,
                    out=rng.choice(["f32", "bf16"]))
    if op == "clip":
        layers = _log(rng, 1, 24)
        return dict(op=op, layers=layers, E=_log(rng, 2, 256), hidden=_log(rng, 16, 4096), inter=_log(rng, 16, 2048),
                    dtype=rng.choice(["f32", "bf16"]) if layers <= 8 else "bf16", below=rng.random() < 0.25)
    return dict(op=op, T=_log(rng, 1, 8192 if op == "train" else 4096), hidden=_mult(rng, 16, 4096, 8),
                inter=_mult(rng, 16, 2048, 8))


def _touched(c):
    """Experts with at least one slot, in expectation (uniform choice)."""
    return min(c["E"], c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"]))


def _shapes(c):
    """Gradients of the layers: router, its bias, norm, both weights of the shared expert."""
    E, H, I = c["E"], c["hidden"], c["inter"]
    return [((E, H), "f32"), ((E,), "f32"), ((H,), "f32"), ((2 * I, H), c["dtype"]), ((H, I), c["dtype"])] * c["layers"]


def work(c):
    op = c["op"]
    if op == "clip":
        n = sum(math.prod(s) * (4 if d == "f32" else 2) for s, d in _shapes(c))
        return {"bytes": 2 * n + 4, "flops": 3 * sum(math.prod(s) for s, _ in _shapes(c))}
    T = c["T"]
    if op in ("decode", "matvec"):
        per = lambda K: K / 2 + K // BLOCK[c["fmt"]]  # noqa: E731
        rows = T * c["k"]
        if op == "matvec":
            return {"bytes": _touched(c) * c["N"] * per(c["K"]) + T * c["K"] * 2 + rows * c["N"] * (4 if c["out"] == "f32" else 2),
                    "flops": 2.0 * rows * c["N"] * c["K"]}
        H, I = c["hidden"], c["inter"]
        return {"bytes": _touched(c) * (2 * I * per(H) + H * per(I)) + T * H * 4 + rows * 8, "flops": 6.0 * rows * H * I}
    H, I = c["hidden"], c["inter"]
    if op == "ffn":
        return {"bytes": 2 * (3 * H * I + 2 * T * H), "flops": 6.0 * T * H * I}
    # x and dout in, out and dx out, the weights in and their gradients out
    return {"bytes": 2 * (6 * H * I + 4 * T * H), "flops": 18.0 * T * H * I}


# ------------------------------------------------------------------- inputs

def _weights4(E, N, K, fmt, g):
    """Uniform codes; block scales over a few binades that keep sums of order one."""
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "mx":
        return codes, torch.randint(114, 122, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8), None
    scales = torch.randint(0x28, 0x41, (E, N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales, 2.0 ** -7 * (1 + torch.randint(0, 8, (E,), generator=g, device="cuda").float() / 8)


def _normal(shape, std, g, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0, std, generator=g)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = c["op"]
    # The status word and scratch a user's program makes once and passes to every call.
    s = dict(case=c, ws=torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"))
    if op == "clip":
        # Flat buffers by type, tensors as consecutive views of them, as trainers keep gradients:
        # behind a tensor of odd length the next one starts off every vector's alignment.
        shapes = _shapes(c)
        flat, out = {}, {}
        for d, dt in (("f32", torch.float32), ("bf16", torch.bfloat16)):
            n = sum(math.prod(s) for s, t in shapes if t == d)
            flat[d] = _normal((n,), 1e-3, g, dt)
            out[d] = torch.empty_like(flat[d])
        at = {"f32": 0, "bf16": 0}
        s["grads"], s["outs"] = [], []
        for shape, d in shapes:
            n = math.prod(shape)
            s["grads"].append(flat[d][at[d]:at[d] + n].view(shape))
            s["outs"].append(out[d][at[d]:at[d] + n].view(shape))
            at[d] += n
        s["flat"], s["flat_out"] = flat, out
        # A norm near the expected one: clipped below it, left as it is above.
        norm = 1e-3 * math.sqrt(sum(math.prod(s) for s, _ in shapes))
        s["max_norm"] = norm * (4.0 if c["below"] else 0.3)
        s["norm"] = torch.empty(1, device="cuda")
        return s
    T = c["T"]
    if op in ("ffn", "train"):
        H, I = c["hidden"], c["inter"]
        s["x"] = _normal((T, H), 1, g)
        s["w13"], s["w2"] = _normal((2 * I, H), H ** -0.5, g), _normal((H, I), I ** -0.5, g)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        s["out"], s["h"] = torch.empty((T, H), **bf), torch.empty((T, I), **bf)
        if op == "train":
            s["dout"] = _normal((T, H), 0.01, g)
            s["gu"], s["dgu"] = torch.empty((T, 2 * I), **bf), torch.empty((T, 2 * I), **bf)
            s["grads"] = (torch.empty((T, H), **bf), torch.empty((2 * I, H), **bf), torch.empty((H, I), **bf))
        return s
    E, k = c["E"], c["k"]
    keys = torch.rand((T, E), generator=g, device="cuda")
    s["ids"] = torch.topk(keys, k, dim=1).indices.to(torch.int32)
    if op == "matvec":
        s["x"] = _normal((T, c["K"]), 1, g)
        s["w"] = _weights4(E, c["N"], c["K"], c["fmt"], g)
        s["y"] = torch.empty((T * k, c["N"]), dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
        return s
    H, I = c["hidden"], c["inter"]
    s["x"] = _normal((T, H), 1, g)
    s["topk_w"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
    s["w13"], s["w2"] = _weights4(E, 2 * I, H, c["fmt"], g), _weights4(E, H, I, c["fmt"], g)
    s["h"] = torch.empty((T * k, I), dtype=torch.bfloat16, device="cuda")
    s["y2"], s["out"] = torch.empty((T * k, H), device="cuda"), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    return s


# -------------------------------------------------------------- plain forms

_tables = {}


def _table(name):
    if name not in _tables:
        mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
        e2m1 = torch.cat([mags, -mags]) + 0.0
        b = torch.arange(256, device="cuda")
        _tables["pairs"] = torch.stack([e2m1[b % 16], e2m1[b // 16]], dim=1)      # low nibble first
        _tables["mx"] = torch.ldexp(torch.ones(256, device="cuda"), (b - 127).float())
        _tables["nv"] = b.to(torch.uint8).view(torch.float8_e4m3fn).float()
    return _tables[name]


def _chosen(w, ids, fmt):
    """float32 weights [slots, N, K] of the slots' experts."""
    codes, scales, ws2 = w
    at = ids.reshape(-1).long()
    v = _table("pairs")[codes[at].int()].flatten(2)
    v = v.unflatten(2, (-1, BLOCK[fmt])) * _table(fmt)[scales[at].int()][..., None]
    return v.flatten(2) if ws2 is None else v.flatten(2) * ws2[at][:, None, None]


def _sigmoid(g):
    return 1 / (1 + torch.exp(-g))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "clip":
        a, b = s["flat"]["f32"], s["flat"]["bf16"]
        norm = (a.square().sum(dtype=torch.float64) + b.float().square().sum(dtype=torch.float64)).sqrt()
        scale = (s["max_norm"] / (norm + 1e-6)).clamp_max(1).float()
        return {"norm": norm.float().view(1), "f32": a * scale, "bf16": (b.float() * scale).to(torch.bfloat16)}
    if op in ("ffn", "train"):
        I = c["inter"]
        x, w13, w2 = s["x"].float(), s["w13"].float(), s["w2"].float()
        g, u = (x @ w13.T).split(I, dim=1)
        sig = _sigmoid(g)
        h = g * sig * u
        out = (h @ w2.T).to(torch.bfloat16)
        if op == "ffn":
            return {"out": out}
        dout = s["dout"].float()
        dh = dout @ w2
        dgu = torch.cat([dh * u * (sig * (1 + g * (1 - sig))), dh * (g * sig)], dim=1)
        return {"out": out, "dx": (dgu @ w13).to(torch.bfloat16), "dw13": (dgu.T @ x).to(torch.bfloat16),
                "dw2": (dout.T @ h).to(torch.bfloat16)}
    fmt, k = c["fmt"], c["k"]
    x = s["x"].float().repeat_interleave(k, dim=0)
    if op == "matvec":
        return {"y": torch.bmm(_chosen(s["w"], s["ids"], fmt), x[:, :, None])[:, :, 0].to(s["y"].dtype)}
    gu = torch.bmm(_chosen(s["w13"], s["ids"], fmt), x[:, :, None])[:, :, 0]
    g, u = gu.split(c["inter"], dim=1)
    y = torch.bmm(_chosen(s["w2"], s["ids"], fmt), (g * _sigmoid(g) * u)[:, :, None])[:, :, 0]
    return {"out": (y.view(c["T"], k, -1) * s["topk_w"][:, :, None]).sum(dim=1).to(torch.bfloat16)}


# -------------------------------------------------------- the library's calls

def _library(s):
    from fp4_weight_grouped_gb300 import binding as B

    c = s["case"]
    op = c["op"]
    if op == "clip":
        norm = B.clip_grads(s["grads"], s["max_norm"], out=s["outs"], norm=s["norm"], workspace=s["ws"])
        return {"norm": norm, "f32": s["flat_out"]["f32"], "bf16": s["flat_out"]["bf16"]}
    if op == "ffn":
        return {"out": B.ffn_forward(s["x"], s["w13"], s["w2"], h=s["h"], out=s["out"], workspace=s["ws"])}
    if op == "train":
        out = B.ffn_forward(s["x"], s["w13"], s["w2"], h=s["h"], gu=s["gu"], out=s["out"], workspace=s["ws"])
        dx, dw13, dw2 = B.ffn_backward(s["dout"], s["x"], s["w13"], s["w2"], s["h"], s["gu"], dgu=s["dgu"],
                                       out=s["grads"], workspace=s["ws"])
        return {"out": out, "dx": dx, "dw13": dw13, "dw2": dw2}
    fmt = B.MOE_FP4_MX if c["fmt"] == "mx" else B.MOE_FP4_NV
    if op == "matvec":
        codes, scales, ws2 = s["w"]
        return {"y": B.fp4_matvec(s["x"], codes, scales, fmt, row_expert=s["ids"].view(-1), index_div=c["k"],
                                  weight_scale_2=ws2, out=s["y"], workspace=s["ws"])}
    out = B.layer_decode(s["x"], s["ids"], s["topk_w"], s["w13"], s["w2"], fmt, h=s["h"], y2=s["y2"], out=s["out"],
                         workspace=s["ws"])
    return {"out": out}


def run(s):
    return _library(s) if own else _plain(s)


# ------------------------------------------------- the definitions in 64 bits

def _x_e2m1(n):
    """e2m1 from its bits: sign, two exponent bits (bias 1), one mantissa bit."""
    e, f = n >> 1 & 3, (n & 1).double()
    mag = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.pow(2.0, (e - 1).double()))
    return torch.where(n >= 8, -mag, mag)


def _x_scale(b, fmt):
    b = b.long()
    if fmt == "mx":
        return torch.pow(torch.full((), 2.0, dtype=torch.float64, device="cuda"), (b - 127).double())
    e, m = b >> 3 & 15, (b & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(b >= 128, -mag, mag)


def _x_matrix(w, e, fmt):
    """Expert e's weights in 64 bits [N, K]."""
    codes, scales, ws2 = w
    b = codes[e].to(torch.int16)
    v = torch.stack([_x_e2m1(b & 15), _x_e2m1(b >> 4)], dim=2).flatten(1)
    v = v * _x_scale(scales[e], fmt).repeat_interleave(BLOCK[fmt], dim=1)
    return v if ws2 is None else v * ws2[e].double()


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "clip":
        norm = torch.sqrt(sum(torch.linalg.vector_norm(g, dtype=torch.float64) ** 2 for g in s["grads"]))
        scale = torch.minimum(s["max_norm"] / (norm + 1e-6), torch.ones_like(norm))
        return {"norm": norm.view(1)} | {d: f.double() * scale for d, f in s["flat"].items()}
    if op in ("ffn", "train"):
        I = c["inter"]
        x, w13, w2 = (s[n].double().requires_grad_(op == "train") for n in ("x", "w13", "w2"))
        y = torch.einsum("th,nh->tn", x, w13)
        out = torch.einsum("ti,hi->th", torch.nn.functional.silu(y[:, :I]) * y[:, I:], w2)
        if op == "ffn":
            return {"out": out}
        out.backward(s["dout"].double())
        return {"out": out.detach(), "dx": x.grad, "dw13": w13.grad, "dw2": w2.grad}
    fmt, k = c["fmt"], c["k"]
    rows = []
    for r, e in enumerate(s["ids"].view(-1).tolist()):
        x = s["x"][r // k].double()
        if op == "matvec":
            rows.append(torch.mv(_x_matrix(s["w"], e, fmt), x))
            continue
        y = torch.mv(_x_matrix(s["w13"], e, fmt), x)
        h = y[:c["inter"]] * torch.sigmoid(y[:c["inter"]]) * y[c["inter"]:]
        rows.append(torch.mv(_x_matrix(s["w2"], e, fmt), h) * s["topk_w"].view(-1)[r].double())
    y = torch.stack(rows)
    return {"y": y} if op == "matvec" else {"out": y.view(c["T"], k, -1).sum(dim=1)}
