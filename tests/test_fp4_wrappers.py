"""What the Python wrappers of the 4-bit path refuse before they call the library, without a
GPU: the library is replaced by a recorder, and the tensors are CPU ones that say they are
CUDA's."""
import pytest
import torch

from fp4_weight_grouped_gb300 import binding as B


class OnGpu(torch.Tensor):
    is_cuda = True


def gpu(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 4096 if name == "moe_workspace_bytes" else 0
        return call


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(B, "load", lambda path=None: r)
    monkeypatch.setattr(B, "_stream", lambda stream=None: 0)
    return r


def layer(T, k, E=4, H=64, I=32, fmt=B.MOE_FP4_MX):
    """Arguments of layer_forward_fp4 but for the buffers."""
    blk = 32 if fmt == B.MOE_FP4_MX else 16
    u8 = torch.uint8
    one = lambda n: gpu((n,), torch.float32)  # noqa: E731
    return (gpu((T, H), torch.bfloat16), gpu((T, k), torch.int32), gpu((T, k), torch.float32),
            (gpu((E, 2 * I, H // 2), u8), gpu((E, 2 * I, H // blk), u8), one(E)),
            (gpu((E, H, I // 2), u8), gpu((E, H, I // blk), u8), one(E)))


def buffers(T, k, E=4, H=64, I=32, fmt=B.MOE_FP4_MX):
    b = B.LayerBuffersFp4(T, k, E, H, I, fmt, device="cpu")
    for name, t in vars(b).items():
        if isinstance(t, torch.Tensor):
            setattr(b, name, t.as_subclass(OnGpu))
    return b


def forward(args, b):
    x2 = gpu((1,), torch.float32)
    return B.layer_forward_fp4(*args, b, x_scale_2=x2, h_scale_2=x2)


@pytest.mark.parametrize("fmt", [B.MOE_FP4_MX, B.MOE_FP4_NV], ids=["mx", "nv"])
def test_layer_takes_its_buffers(lib, fmt):
    b = buffers(4, 2, fmt=fmt)
    assert forward(layer(4, 2, fmt=fmt), b) is b.out
    assert lib.calls[-1] == "moe_layer_forward_fp4"


def test_layer_refuses_buffers_of_fewer_tokens(lib):
    """T and k exchanged: the same rows, but out holds T of them."""
    with pytest.raises(ValueError, match="out"):
        forward(layer(8, 1), buffers(4, 2))
    assert "moe_layer_forward_fp4" not in lib.calls


@pytest.mark.parametrize("fmt", [B.MOE_FP4_MX, B.MOE_FP4_NV], ids=["mx", "nv"])
@pytest.mark.parametrize("name", ["out", "y2", "x_codes", "x_scales", "h_codes", "h_scales", "group_sizes",
                                  "group_offsets", "sorted_slot", "slot_to_row"])
def test_layer_refuses_a_wrong_buffer(lib, name, fmt):
    for change in (lambda t: t[:-1].contiguous(), lambda t: t.to(torch.float64), lambda t: t.as_subclass(torch.Tensor)):
        b = buffers(4, 2, fmt=fmt)
        setattr(b, name, change(getattr(b, name)))
        with pytest.raises(ValueError, match=name):
            forward(layer(4, 2, fmt=fmt), b)
    assert "moe_layer_forward_fp4" not in lib.calls


@pytest.mark.parametrize("fmt", [B.MOE_FP4_MX, B.MOE_FP4_NV], ids=["mx", "nv"])
def test_layer_takes_larger_buffers(lib, fmt):
    """One set of buffers serves every batch that fits: the first T rows of out are the result."""
    b = buffers(8, 2, fmt=fmt)
    for T, k in ((1, 2), (7, 2), (8, 1), (5, 3)):
        out = forward(layer(T, k, fmt=fmt), b)
        assert out.shape == (T, 64) and out.data_ptr() == b.out.data_ptr()
        assert lib.calls[-1] == "moe_layer_forward_fp4"
    lib.calls.clear()
    for T, k in ((9, 1), (6, 3)):
        with pytest.raises(ValueError):
            forward(layer(T, k, fmt=fmt), b)
    assert "moe_layer_forward_fp4" not in lib.calls


class Side:
    """In place of torch.cuda.Stream."""

    def __init__(self, handle=4096):
        self.cuda_stream = handle

    def __eq__(self, other):
        return isinstance(other, Side) and self.cuda_stream == other.cuda_stream


class Foreign:
    """Another library's stream: a handle alone."""
    cuda_stream = 4096


class Streams:
    """In place of torch.cuda.stream: which stream is current where."""

    def __init__(self, monkeypatch):
        self.now, self.made = None, []
        empty = torch.empty
        monkeypatch.setattr(torch.cuda, "Stream", Side)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Side(handle))
        monkeypatch.setattr(torch.cuda, "stream", self.enter)
        monkeypatch.setattr(torch, "empty", lambda *a, **kw: (self.made.append(self.now), empty(*a, **kw))[1])

    def enter(self, stream):
        import contextlib

        @contextlib.contextmanager
        def on():
            was, self.now = self.now, stream
            yield
            self.now = was
        return on()


def test_what_a_wrapper_makes_belongs_to_the_calls_stream(lib, monkeypatch):
    """A workspace made on the current stream for a call on another one goes back to the
    current stream's pool at return, while that call may still clear and write it; and memory
    that the current stream still uses may become an output that the other one writes."""
    x = gpu((4, 64), torch.float32)
    codes, scales = gpu((4, 32), torch.uint8), gpu((4, 2), torch.uint8)
    w, wsc, sizes = gpu((2, 64, 32), torch.uint8), gpu((2, 64, 2), torch.uint8), gpu((2,), torch.int32)
    s2r, tw = gpu((8,), torch.int32), gpu((4, 2), torch.float32)
    monkeypatch.setattr(B, "_need", lambda *a: None)      # what torch.empty gives here is a CPU tensor
    side = Side()
    calls = {
        "gate": lambda s: B.topk_gate(x, 2, stream=s),
        "gate backward": lambda s: B.topk_gate_backward(x, gpu((4, 2), torch.int32), tw, stream=s),
        "quantise": lambda s: B.fp4_quantize(x, B.MOE_FP4_MX, stream=s),
        "product": lambda s: B.fp4_grouped_gemm(codes, scales, w, wsc, sizes, B.MOE_FP4_MX, stream=s),
        "swiglu": lambda s: B.fp4_grouped_gemm_swiglu(codes, scales, w, wsc, sizes, B.MOE_FP4_MX, stream=s),
        "combine": lambda s: B.combine_backward(x, gpu((8, 64), torch.float32), s2r, tw, stream=s),
        "gather": lambda s: B.gather_backward(gpu((8, 64), torch.float32), s2r, 2, stream=s),
        "workspace": lambda s: B.make_workspace(4, 2, 4, "cpu", s),
    }
    seen = Streams(monkeypatch)
    for name, call in calls.items():
        for stream, want in ((side, side), (Foreign(), side), (None, None)):
            seen.made.clear()
            call(stream)
            assert seen.made and all(s == want for s in seen.made), (name, seen.made)


def test_a_workspace_the_kernels_cannot_write_is_refused(lib):
    x, sizes = gpu((4, 64), torch.float32), gpu((2,), torch.int32)
    codes, scales = gpu((4, 32), torch.uint8), gpu((4, 2), torch.uint8)
    w, wsc = gpu((2, 64, 32), torch.uint8), gpu((2, 64, 2), torch.uint8)
    ops = (codes, scales, w, wsc, sizes, B.MOE_FP4_MX)
    b = buffers(4, 2)
    good = gpu((256,), torch.uint8)
    out = dict(gemm=gpu((4, 64), torch.float32), h=(gpu((4, 16), torch.uint8), gpu((4, 1), torch.uint8)))
    calls = {
        "moe_fp4_quantize": lambda ws: B.fp4_quantize(x, B.MOE_FP4_MX, out=(codes, scales), workspace=ws),
        "moe_fp4_grouped_gemm": lambda ws: B.fp4_grouped_gemm(*ops, out=out["gemm"], workspace=ws),
        "moe_fp4_grouped_gemm_swiglu": lambda ws: B.fp4_grouped_gemm_swiglu(*ops, out=out["h"], workspace=ws),
        "moe_layer_forward_fp4": lambda ws: (setattr(b, "workspace", ws), forward(layer(4, 2), b)),
    }
    for name, call in calls.items():
        call(good)
        assert lib.calls[-1] == name
        lib.calls.clear()
        for bad in (torch.zeros(4096, dtype=torch.uint8), gpu((8192,), torch.uint8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)
        assert name not in lib.calls


def test_layer_refuses_results_of_another_width(lib):
    """out may have more rows than the call, not other ones."""
    for shape in ((8, 32), (4, 128), (256,), (4, 1, 64)):
        b = buffers(4, 2)
        b.out = gpu(shape, torch.float32)
        with pytest.raises(ValueError, match="out"):
            forward(layer(4, 2), b)
    assert "moe_layer_forward_fp4" not in lib.calls
