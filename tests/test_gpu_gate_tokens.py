"""The router gate at as many tokens as its interface takes: T * k = 2^31 - 1."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


def test_every_token_count_of_the_interface(B):
    T = 2 ** 31 - 1
    logits = torch.full((1, 1), 0.25, dtype=torch.bfloat16, device="cuda").expand(T, 1)     # row stride 0
    ids = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), -1.0, device="cuda")
    B.topk_gate(logits, 1, out=(ids, w))
    assert int(ids.min()) == 0 and int(ids.max()) == 0
    assert float(w.min()) == 1.0 and float(w.max()) == 1.0
    dl = torch.full((T, 1), 5.0, dtype=torch.bfloat16, device="cuda")
    B.topk_gate_backward(logits, ids, w, out=dl)
    assert float(dl.min()) == 0.0 and float(dl.max()) == 0.0       # one expert: its weight is constant
