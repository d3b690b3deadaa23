"""Sizes past 32 bits in the Python wrappers of the few-row products and the dense block, without
a GPU: the library is replaced by a recorder, and the tensors are ones without memory that say they
are on CUDA device 0.  Handed on by its lower 32 bits a size passes the library's checks as a
smaller one: rows of x past its end are read, or rows of the output are not written."""
import pytest
import torch

from fp4_weight_grouped_gb300 import binding as B

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
WRAP = 2 ** 32


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def gpu(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: made.append((name, args)) or 0

    monkeypatch.setattr(B, "load", lambda path=None: Recorder())
    monkeypatch.setattr(B, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    return made


WS = gpu((4096,), U8)


def matvec(f, rows=6, x_rows=3, K=64, N=48, E=4, div=2, ids=True):
    n = N // 2 if f is B.fp4_matvec_swiglu else N
    return f(gpu((x_rows, K), BF), gpu((E, N, K // 2), U8), gpu((E, N, K // 32), U8), B.MOE_FP4_MX,
             row_expert=gpu((rows,), I32) if ids else None, index_div=div, out=gpu((rows, n), BF), workspace=WS)


@pytest.mark.parametrize("f", [B.fp4_matvec, B.fp4_matvec_swiglu], ids=["plain", "swiglu"])
def test_matvec(calls, f):
    matvec(f)
    assert len(calls) == 1
    for bad in (dict(div=WRAP + 1), dict(div=WRAP + 1, rows=3 * WRAP + 3, ids=False), dict(rows=WRAP + 6, x_rows=WRAP // 2 + 3),
                dict(K=WRAP + 64), dict(N=WRAP + 48), dict(E=WRAP + 4), dict(div=2 ** 31)):
        with pytest.raises(ValueError, match="32 bits"):
            matvec(f, **bad)
    assert len(calls) == 1


def decode(T=3, k=2, E=4, hidden=64, inter=32):
    return B.layer_decode(gpu((T, hidden), BF), gpu((T, k), I32), gpu((T, k), F32),
                          (gpu((E, 2 * inter, hidden // 2), U8), gpu((E, 2 * inter, hidden // 32), U8), None),
                          (gpu((E, hidden, inter // 2), U8), gpu((E, hidden, inter // 32), U8), None), B.MOE_FP4_MX,
                          h=gpu((T * k, inter), BF), y2=gpu((T * k, hidden), F32), out=gpu((T, hidden), BF), workspace=WS)


def test_layer_decode(calls):
    decode()
    assert len(calls) == 1
    for bad in (dict(T=WRAP + 3), dict(k=WRAP + 2), dict(E=WRAP + 4), dict(hidden=WRAP + 64), dict(inter=WRAP + 32)):
        with pytest.raises(ValueError, match="32 bits"):
            decode(**bad)
    assert len(calls) == 1


def ffn(T=5, hidden=64, inter=24, back=False):
    x, w13, w2, h, gu = (gpu(s, BF) for s in ((T, hidden), (2 * inter, hidden), (hidden, inter), (T, inter), (T, 2 * inter)))
    if not back:
        return B.ffn_forward(x, w13, w2, h=h, gu=gu, out=gpu((T, hidden), BF), workspace=WS)
    return B.ffn_backward(gpu((T, hidden), BF), x, w13, w2, h, gu, dgu=gpu((T, 2 * inter), BF),
                          out=(gpu((T, hidden), BF), gpu((2 * inter, hidden), BF), gpu((hidden, inter), BF)), workspace=WS)


@pytest.mark.parametrize("back", [False, True], ids=["forward", "backward"])
def test_ffn(calls, back):
    ffn(back=back)
    assert len(calls) == 1
    for bad in (dict(T=WRAP + 5), dict(T=WRAP), dict(hidden=WRAP + 64), dict(inter=WRAP + 24)):
        with pytest.raises(ValueError, match="32 bits"):
            ffn(**bad, back=back)
    assert len(calls) == 1
