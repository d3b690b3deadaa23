"""What the Python wrappers of the few-row products, the dense block and the clipping refuse
before they call the library, without a GPU: the library is replaced by a recorder, and the
tensors are CPU ones that say they are on CUDA device 0."""
import pytest
import torch

from fp4_weight_grouped_gb300 import binding as B

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


class Elsewhere(OnGpu):
    def get_device(self):
        return 1


def gpu(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 256 if name == "moe_workspace_bytes" else 0
        return call


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(B, "load", lambda path=None: r)
    monkeypatch.setattr(B, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    return r


WS = gpu((B.MOE_GRAD_WORKSPACE_BYTES,), U8)


def matvec():
    return dict(x=gpu((3, 64), BF), codes=gpu((4, 48, 32), U8), scales=gpu((4, 48, 2), U8), fmt=B.MOE_FP4_MX,
                row_expert=gpu((6,), I32), index_div=2, out=gpu((6, 48), F32), workspace=WS)


def ffn():
    return dict(x=gpu((5, 64), BF), w13=gpu((48, 64), BF), w2=gpu((64, 24), BF), h=gpu((5, 24), BF), gu=gpu((5, 48), BF),
                out=gpu((5, 64), BF), workspace=WS)


def back():
    return dict(dout=gpu((5, 64), BF), x=gpu((5, 64), BF), w13=gpu((48, 64), BF), w2=gpu((64, 24), BF), h=gpu((5, 24), BF),
                gu=gpu((5, 48), BF), dgu=gpu((5, 48), BF),
                out=(gpu((5, 64), BF), gpu((48, 64), F32), gpu((64, 24), F32)), workspace=WS)


def decode():
    return dict(x=gpu((3, 64), BF), topk_ids=gpu((3, 2), I32), topk_w=gpu((3, 2), F32),
                w13=(gpu((4, 64, 32), U8), gpu((4, 64, 2), U8), None), w2=(gpu((4, 64, 16), U8), gpu((4, 64, 1), U8), None),
                fmt=B.MOE_FP4_MX, h=gpu((6, 32), BF), y2=gpu((6, 64), F32), out=gpu((3, 64), BF), workspace=WS)


def swiglu():
    return {**matvec(), "out": gpu((6, 24), BF)}


CALLS = {"moe_fp4_matvec": (B.fp4_matvec, matvec), "moe_fp4_matvec_swiglu": (B.fp4_matvec_swiglu, swiglu),
         "moe_ffn_forward": (B.ffn_forward, ffn), "moe_ffn_backward": (B.ffn_backward, back),
         "moe_layer_decode": (B.layer_decode, decode)}


def changed(value):
    """Wrong versions of an argument: a type, a size, gaps, no CUDA memory, another device."""
    if isinstance(value, tuple):
        for i, v in enumerate(value):
            for w in changed(v):
                yield (*value[:i], w, *value[i + 1:])
        return
    if not isinstance(value, torch.Tensor):
        return
    yield value.as_subclass(torch.Tensor).to(torch.float64).as_subclass(OnGpu)
    yield value[:-1].contiguous()
    yield value.as_subclass(torch.Tensor)
    yield value.as_subclass(Elsewhere)
    if value.dim() > 1:
        yield torch.zeros((*value.shape[:-1], 2 * value.shape[-1]), dtype=value.dtype).as_subclass(OnGpu)[..., ::2]


@pytest.mark.parametrize("name", CALLS)
def test_calls_and_refusals(lib, name):
    f, make = CALLS[name]
    good = make()
    f(**good)
    assert lib.calls[-1][0] == name
    for key, value in good.items():
        if key == "workspace":
            continue
        for wrong in changed(value):
            lib.calls.clear()
            with pytest.raises(ValueError):
                f(**{**good, key: wrong})
            assert not [c for c in lib.calls if c[0] == name], key


@pytest.mark.parametrize("name", CALLS)
def test_a_workspace_the_kernels_cannot_write_is_refused(lib, name):
    f, make = CALLS[name]
    for bad in (torch.zeros(4096, dtype=U8), gpu((8192,), U8)[::2], torch.zeros(4096, dtype=U8).as_subclass(Elsewhere)):
        with pytest.raises(ValueError):
            f(**{**make(), "workspace": bad})
    assert not [c for c in lib.calls if c[0] == name]


def test_rows_that_x_does_not_have_are_refused(lib):
    a = matvec()
    for change in (dict(row_expert=gpu((7,), I32), out=gpu((7, 48), F32)), dict(index_div=1), dict(index_div=0)):
        with pytest.raises(ValueError):
            B.fp4_matvec(**{**a, **change})
    B.fp4_matvec(**{**a, "row_expert": gpu((5,), I32), "out": gpu((5, 48), F32)})      # a last token of fewer rows
    assert lib.calls[-1][0] == "moe_fp4_matvec"
    B.fp4_matvec(**{**a, "row_expert": None})                                         # every row of x, index_div times
    assert lib.calls[-1][1][4] == 6


def test_nvfp4_needs_its_tensor_scales(lib):
    a = {**matvec(), "fmt": B.MOE_FP4_NV, "scales": gpu((4, 48, 4), U8)}
    for g in (None, gpu((3,), F32), gpu((4,), BF)):
        with pytest.raises(ValueError):
            B.fp4_matvec(**a, weight_scale_2=g)
    B.fp4_matvec(**a, weight_scale_2=gpu((4,), F32))
    with pytest.raises(ValueError):
        B.fp4_matvec(**{**a, "fmt": 7}, weight_scale_2=gpu((4,), F32))


def test_an_odd_number_of_gate_and_up_rows_is_refused(lib):
    with pytest.raises(ValueError, match="odd"):
        B.fp4_matvec_swiglu(**{**swiglu(), "codes": gpu((4, 47, 32), U8), "scales": gpu((4, 47, 2), U8)})


def test_backward_leaves_out_what_is_none(lib):
    a = back()
    for i in range(3):
        out = list(a["out"])
        out[i] = None
        B.ffn_backward(**{**a, "out": tuple(out)})
        args = lib.calls[-1][1]
        assert [p is None for p in args[11:14]] == [j == i for j in range(3)]
    with pytest.raises(ValueError, match="one type"):
        B.ffn_backward(**{**a, "out": (a["out"][0], a["out"][1], gpu((64, 24), BF))})


def test_clipping(lib):
    g = [gpu((3, 4), F32), gpu((7,), BF), gpu((0,), F32)]
    norm = gpu((1,), F32)
    ok = dict(norm=norm, workspace=WS)
    assert B.clip_grads(g, 1.0, **ok) is norm
    assert B.clip_grads(tuple(g), 1.0, out=[t.clone() for t in g], **ok) is norm
    assert B.grad_norm(g, **ok) is norm
    bad = [torch.zeros((3, 4), dtype=torch.float64).as_subclass(OnGpu), torch.zeros((3, 4)), gpu((3, 8), F32)[:, ::2],
           torch.zeros((3, 4)).as_subclass(Elsewhere), gpu((3, 4), torch.float16)]
    lib.calls.clear()
    for t in bad:
        for call in (lambda: B.clip_grads([g[1], t], 1.0, **ok), lambda: B.grad_norm([t], **ok),
                     lambda: B.clip_grads([g[0]], 1.0, out=[t], **ok)):
            with pytest.raises(ValueError):
                call()
    for out in ([g[0]], [g[1], g[0], g[2]], [g[0], g[1], gpu((1,), F32)]):
        with pytest.raises(ValueError):
            B.clip_grads(g, 1.0, out=out, **ok)
    for n in (gpu((2,), F32), gpu((1,), BF), torch.zeros(1)):
        with pytest.raises(ValueError):
            B.clip_grads(g, 1.0, norm=n, workspace=WS)
    assert not lib.calls


def test_decode_takes_larger_intermediates(lib):
    a = decode()
    B.layer_decode(**{**a, "h": gpu((64, 32), BF), "y2": gpu((64, 64), F32)})
    assert lib.calls[-1][0] == "moe_layer_decode"
