"""Host checks of the 4-bit, gate and gradient entry points through the C ABI, without a
GPU: only calls that are rejected before any device work are made (the pointers are
not device memory)."""
import ctypes as C

import pytest

from fp4_weight_grouped_gb300 import binding, build_lib

P = C.c_void_p
OK, INVALID = 0, 1
FAKE, ODD = 4096, 4100          # aligned to 16 bytes, and to 4 only


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


def check(f, good, bad):
    """Every change in `bad` makes the good call invalid."""
    names = list(good)
    for change in bad:
        assert set(change) <= set(names), change
        args = [{**good, **change}[n] for n in names]
        assert f(*args) == INVALID, change


GATE = dict(logits=FAKE, dtype=0, stride=64, T=8, E=64, k=6, renorm=0, ids=FAKE, w=FAKE, stream=None)
GATE_BAD = [dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(dtype=2), dict(stride=-1),
            dict(logits=None), dict(logits=4098), dict(ids=None), dict(w=None), dict(T=2 ** 30, k=6)]


def test_gate(lib):
    check(lib.moe_topk_gate, GATE, GATE_BAD)
    good = {**{n: v for n, v in GATE.items() if n not in ("w", "stream")}, "dw": FAKE, "dl": FAKE, "stream": None}
    bad = [b for b in GATE_BAD if "w" not in b] + [dict(dw=None), dict(dl=None), dict(dl=4098)]
    check(lib.moe_topk_gate_backward, good, bad)


QUANT = dict(x=FAKE, dtype=1, x_rows=8, x_stride=64, K=64, index=None, div=1, rows=8, fmt=0, ts=None, codes=FAKE,
             scales=FAKE, values=None, vdt=0, ws=FAKE, wsb=256, stream=None)


def test_quantize(lib):
    check(lib.moe_fp4_quantize, QUANT,
          [dict(dtype=2), dict(fmt=2), dict(K=0), dict(K=48), dict(x_rows=-1), dict(x_stride=-1), dict(rows=-1),
           dict(rows=9), dict(div=0), dict(index=FAKE, div=0), dict(fmt=1), dict(fmt=1, ts=4098), dict(codes=None),
           dict(codes=ODD), dict(scales=None), dict(x=None), dict(x=4097), dict(dtype=0, x=4098),
           dict(values=FAKE, vdt=3), dict(values=ODD), dict(ws=None), dict(wsb=255), dict(ws=ODD)])


GEMM = dict(ac=FAKE, asc=FAKE, a2=None, rows=8, K=64, wc=FAKE, wsc=FAKE, w2=None, fmt=0, sizes=FAKE, E=4, N=128,
            out=FAKE, dt=0, ws=FAKE, wsb=256, stream=None)
GEMM_BAD = [dict(rows=-1), dict(rows=2 ** 31 - 1), dict(K=0), dict(K=40), dict(E=0), dict(E=1025), dict(ac=None),
            dict(ac=ODD), dict(asc=None), dict(wc=None), dict(wc=ODD), dict(wsc=None), dict(sizes=None), dict(fmt=5),
            dict(fmt=1), dict(fmt=1, a2=FAKE), dict(fmt=1, w2=FAKE), dict(fmt=1, a2=4098, w2=FAKE), dict(ws=None),
            dict(ws=ODD), dict(wsb=10)]


def test_products(lib):
    check(lib.moe_fp4_grouped_gemm, GEMM,
          GEMM_BAD + [dict(N=0), dict(E=1024, N=2 ** 21), dict(out=None), dict(out=4098), dict(dt=1, out=4097), dict(dt=7)])
    good = {**{n: v for n, v in GEMM.items() if n not in ("N", "out", "dt", "ws", "wsb", "stream")}, "I": 64, "h2": None,
            "hc": FAKE, "hs": FAKE, "ws": FAKE, "wsb": 256, "stream": None}
    check(lib.moe_fp4_grouped_gemm_swiglu, good,
          GEMM_BAD + [dict(I=0), dict(I=48), dict(E=1024, I=2 ** 20), dict(hc=None), dict(hc=ODD), dict(hs=None),
                      dict(fmt=1, a2=FAKE, w2=FAKE)])


def test_layer(lib):
    good = dict(x=FAKE, ids=FAKE, w=FAKE, T=8, k=2, E=4, hidden=64, inter=32, fmt=0, c13=FAKE, s13=FAKE, g13=None,
                c2=FAKE, s2=FAKE, g2=None, xs2=None, hs2=None, out=FAKE, gs=FAKE, off=FAKE, ss=FAKE, s2r=FAKE, xc=FAKE,
                xs=FAKE, hc=FAKE, hs=FAKE, y2=FAKE, ws=FAKE, wsb=1 << 20, stream=None)
    check(lib.moe_layer_forward_fp4, good,
          [dict(hidden=0), dict(hidden=48), dict(inter=16), dict(T=-1), dict(k=5), dict(E=0), dict(fmt=3), dict(fmt=1)] +
          [{n: None} for n in ("x", "ids", "w", "c13", "s13", "c2", "s2", "out", "gs", "off", "ss", "s2r", "xc", "xs",
                               "hc", "hs", "y2", "ws")] +
          [dict(out=ODD), dict(y2=ODD), dict(xc=ODD), dict(hc=ODD), dict(c13=ODD), dict(wsb=300)])


def test_gradients(lib):
    good = dict(dout=FAKE, ddt=0, y=FAKE, ydt=0, s2r=FAKE, w=FAKE, T=8, k=2, N=64, dy=FAKE, dydt=0, dw=FAKE, stream=None)
    check(lib.moe_combine_backward, good,
          [dict(T=-1), dict(k=0), dict(N=0), dict(T=2 ** 30, k=4), dict(ddt=2), dict(ydt=2), dict(dydt=2), dict(dout=None),
           dict(s2r=None), dict(w=None), dict(y=None), dict(dy=None, dw=None), dict(dout=ODD), dict(y=ODD), dict(dy=ODD)])
    good = dict(dxs=FAKE, idt=0, s2r=FAKE, T=8, k=2, hidden=64, dx=FAKE, odt=0, stream=None)
    check(lib.moe_gather_backward, good,
          [dict(T=-1), dict(k=0), dict(hidden=0), dict(T=2 ** 30, k=4), dict(idt=3), dict(odt=3), dict(dxs=None),
           dict(s2r=None), dict(dx=None), dict(dxs=ODD), dict(dx=ODD)])
