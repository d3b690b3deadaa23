"""Host checks of the few-row products, the dense block and the gradient clipping through the
C ABI, without a GPU: only calls that are rejected before any device work are made (the
pointers are not device memory)."""
import ctypes as C

import pytest

from fp4_weight_grouped_gb300 import binding, build_lib

OK, INVALID, UNSUPPORTED, CUDA, CAPACITY = 0, 1, 2, 3, 6
FAKE, ODD = 4096, 4100          # aligned to 16 bytes, and to 4 only


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


def check(f, good, bad, status=INVALID):
    """Every change in `bad` makes the good call invalid."""
    for change in bad:
        assert set(change) <= set(good), change
        args = {**good, **change}
        assert f(*args.values()) == status, change


MATVEC = dict(x=FAKE, x_stride=64, div=2, ids=FAKE, rows=6, K=64, codes=FAKE, scales=FAKE, ws2=None, fmt=0, E=4, N=48,
              out=FAKE, dt=0, ws=FAKE, wsb=256, stream=None)
MATVEC_BAD = [dict(x=None), dict(x=4097), dict(x_stride=-1), dict(div=0), dict(rows=-1), dict(K=0), dict(K=48),
              dict(codes=None), dict(codes=ODD), dict(scales=None), dict(fmt=2), dict(fmt=1), dict(fmt=1, ws2=4098),
              dict(E=0), dict(E=1025), dict(ws=None), dict(ws=ODD), dict(wsb=255)]


def test_matvec(lib):
    check(lib.moe_fp4_matvec, MATVEC,
          MATVEC_BAD + [dict(N=0), dict(E=1024, N=2 ** 21), dict(rows=512, N=2 ** 22), dict(out=None), dict(out=4098),
                        dict(dt=1, out=4097), dict(dt=2)])
    check(lib.moe_fp4_matvec, MATVEC, [dict(rows=513), dict(K=32768 + 32)], CAPACITY)
    good = {**{n: v for n, v in MATVEC.items() if n not in ("N", "out", "dt", "ws", "wsb", "stream")}, "I": 24, "h": FAKE,
            "ws": FAKE, "wsb": 256, "stream": None}
    check(lib.moe_fp4_matvec_swiglu, good,
          MATVEC_BAD + [dict(I=0), dict(E=1024, I=2 ** 20), dict(h=None), dict(h=4097)])
    check(lib.moe_fp4_matvec_swiglu, good, [dict(rows=513), dict(K=32768 + 32)], CAPACITY)


def test_layer_decode(lib):
    good = dict(x=FAKE, ids=FAKE, w=FAKE, T=3, k=2, E=4, hidden=64, inter=32, fmt=0, c13=FAKE, s13=FAKE, g13=None, c2=FAKE,
                s2=FAKE, g2=None, h=FAKE, y2=FAKE, out=FAKE, dt=0, ws=FAKE, wsb=256, stream=None)
    check(lib.moe_layer_decode, good,
          [dict(T=-1), dict(k=0), dict(E=0), dict(E=1025), dict(hidden=0), dict(hidden=48), dict(inter=0), dict(inter=16),
           dict(fmt=3), dict(fmt=1), dict(fmt=1, g13=FAKE), dict(fmt=1, g2=FAKE), dict(dt=2), dict(T=2 ** 30, k=1000),
           dict(wsb=255)] +
          [{n: None} for n in ("x", "ids", "w", "c13", "s13", "c2", "s2", "h", "y2", "out", "ws")] +
          [dict(out=4098), dict(y2=4098), dict(h=4097), dict(c13=ODD), dict(c2=ODD), dict(ws=ODD)])
    # an invalid argument of either product comes before a capacity of the other
    check(lib.moe_layer_decode, good, [dict(T=300), dict(hidden=65536), dict(inter=65536)], CAPACITY)
    check(lib.moe_layer_decode, good, [dict(T=300, c2=None), dict(hidden=65536, inter=40)])


def test_ids_and_weights_off_their_alignment(lib):
    """A load of four bytes at another address would end the process's use of the GPU."""
    good = {**{n: v for n, v in MATVEC.items() if n not in ("N", "out", "dt", "ws", "wsb", "stream")}, "I": 24, "h": FAKE,
            "ws": FAKE, "wsb": 256, "stream": None}
    for ids in (4097, 4098):
        check(lib.moe_fp4_matvec, {**MATVEC, "rows": 513}, [dict(ids=ids)])
        check(lib.moe_fp4_matvec_swiglu, {**good, "rows": 513}, [dict(ids=ids)])
    good = dict(x=FAKE, ids=FAKE, w=FAKE, T=300, k=2, E=4, hidden=64, inter=32, fmt=0, c13=FAKE, s13=FAKE, g13=None, c2=FAKE,
                s2=FAKE, g2=None, h=FAKE, y2=FAKE, out=FAKE, dt=0, ws=FAKE, wsb=256, stream=None)
    check(lib.moe_layer_decode, good, [dict(ids=4098), dict(w=4097), dict(w=4098)])


FFN = dict(x=FAKE, x_stride=72, T=5, hidden=64, inter=32, w13=FAKE, w2=FAKE, gu=FAKE, h=FAKE, out=FAKE, dt=1, ws=FAKE,
           wsb=256, stream=None)
FFN_BAD = [dict(x=None), dict(x=FAKE + 8), dict(x_stride=56), dict(x_stride=68), dict(x_stride=-8), dict(T=-1),
           dict(T=2 ** 30), dict(hidden=0), dict(hidden=60), dict(hidden=-8), dict(inter=0), dict(inter=4),
           dict(inter=2 ** 29), dict(w13=None), dict(w13=ODD), dict(w2=None), dict(w2=ODD), dict(gu=ODD), dict(h=ODD),
           dict(ws=None), dict(ws=ODD), dict(wsb=255)]


def test_ffn(lib):
    check(lib.moe_ffn_forward, FFN, FFN_BAD + [dict(h=None), dict(out=None), dict(out=ODD), dict(dt=2)])
    good = dict(dout=FAKE, x=FAKE, x_stride=72, T=5, hidden=64, inter=32, w13=FAKE, w2=FAKE, h=FAKE, gu=FAKE, dgu=FAKE,
                dx=FAKE, dw13=FAKE, dw2=FAKE, dt=1, ws=FAKE, wsb=256, stream=None)
    check(lib.moe_ffn_backward, good,
          FFN_BAD + [dict(dout=None), dict(dout=ODD), dict(h=None), dict(gu=None), dict(dgu=None), dict(dgu=ODD),
                     dict(dx=ODD), dict(dw13=ODD), dict(dw2=ODD), dict(dt=2), dict(dx=None, gu=None),
                     dict(dw13=None, dgu=None)])


def grads(sizes, dtypes, ptrs=None, outs=None):
    n = len(sizes)
    ptrs = ptrs or [FAKE + (i << 24) for i in range(n)]
    return ((C.c_uint64 * n)(*ptrs), (C.c_int64 * n)(*sizes), (C.c_int32 * n)(*dtypes), n,
            None if outs is None else (C.c_uint64 * n)(*outs))


def test_gradients(lib):
    p, s, d, n, _ = grads([10, 20], [0, 1])
    a = C.addressof
    good = dict(p=a(p), s=a(s), d=a(d), n=n, norm=FAKE, ws=FAKE, wsb=32768, stream=None)
    bad = [dict(n=-1), dict(p=None), dict(s=None), dict(d=None), dict(norm=None), dict(norm=4098), dict(ws=None),
           dict(ws=ODD), dict(wsb=32767)]
    check(lib.moe_grad_norm, good, bad)
    clip = dict(p=a(p), s=a(s), d=a(d), n=n, most=1.0, eps=0.0, outs=None, norm=FAKE, ws=FAKE, wsb=32768, stream=None)
    inf, nan = float("inf"), float("nan")
    check(lib.moe_grad_clip, clip, bad + [dict(most=-1.0), dict(most=nan), dict(eps=-1.0), dict(eps=nan), dict(eps=inf)])
    for sizes, dtypes, ptrs, outs in (([-1], [0], None, None), ([10], [2], None, None), ([10], [0], [4098], None),
                                      ([10], [1], [4097], None), ([10], [0], [0], None), ([2 ** 62], [0], None, None),
                                      ([10], [0], None, [0]), ([10], [0], None, [4098]),
                                      # the same memory twice, in place; an output over another's input or output
                                      ([10, 10], [0, 0], [FAKE, FAKE], None), ([10, 10], [0, 0], [FAKE, FAKE + 36], None),
                                      ([10, 10], [1, 1], [FAKE + 18, FAKE], None),
                                      ([10, 10], [0, 0], [FAKE, 8192], [16384, 16384]),
                                      ([10, 10], [0, 0], [FAKE, 8192], [8192, 16384]),
                                      ([10], [0], [FAKE], [FAKE + 4])):
        p, s, d, n, o = grads(sizes, dtypes, ptrs, outs)
        assert lib.moe_grad_clip(a(p), a(s), a(d), n, 1.0, 0.0, None if o is None else a(o), FAKE, FAKE, 32768, None) == INVALID
    # neighbours, exchanged order, nothing in between, the same gradient read twice: these pass the
    # checks and stop at the device, where there is none
    import torch
    if torch.cuda.is_available():
        return
    for sizes, dtypes, ptrs, outs in (([10, 10], [0, 0], [FAKE + 40, FAKE], None), ([10, 0, 10], [0, 0, 0], [FAKE, 0, FAKE + 40], None),
                                      ([10, 10], [0, 0], [FAKE, FAKE], [8192, 16384]),
                                      ([10, 10], [0, 0], [FAKE, 8192], [FAKE, 16384])):
        p, s, d, n, o = grads(sizes, dtypes, ptrs, outs)
        assert lib.moe_grad_clip(a(p), a(s), a(d), n, 1.0, 0.0, None if o is None else a(o), FAKE, FAKE, 32768,
                                 None) in (UNSUPPORTED, CUDA)
