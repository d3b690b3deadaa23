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
