"""What the wrappers of the gradient norm and the clipping take as a list, without a GPU: the
library is replaced by a recorder, and the tensors are CPU ones that say they are on CUDA device 0."""
import ctypes as C

import pytest
import torch

from fp4_weight_grouped_gb300 import binding as B


class OnGpu(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def gpu(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Recorder:
        def __getattr__(self, name):
            def call(*args):
                n = args[3]
                made.append((name, n, list((C.c_int64 * n).from_address(args[1]))))
                return 0
            return call

    monkeypatch.setattr(B, "load", lambda path=None: Recorder())
    monkeypatch.setattr(B, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_empty", lambda shape, dtype, device, stream: gpu(shape, dtype))
    return made


@pytest.mark.parametrize("kind", [list, tuple, iter, lambda t: dict(enumerate(t)).values(), lambda t: (x for x in t)],
                         ids=["list", "tuple", "iterator", "values", "generator"])
def test_any_iterable_of_gradients(calls, kind):
    """The norm's tensor and the workspace are made from the first gradient's device, behind the
    arrays that the library reads: by then an iterator is used up."""
    g = [gpu((3, 4), torch.float32), gpu((7,), torch.bfloat16)]
    B.grad_norm(kind(g))
    B.clip_grads(kind(g), 1.0)
    B.clip_grads(kind(g), 1.0, out=kind([t.clone() for t in g]))
    assert calls == [("moe_grad_norm", 2, [12, 7])] + [("moe_grad_clip", 2, [12, 7])] * 2
