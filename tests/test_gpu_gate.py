"""Router gate (moe_topk_gate) and its gradient against plain 64-bit forms.

Tolerances, fixed before the first run.  ids: exact (a stable descending sort).
Weights: e^(v - m) carries the rounding of v - m (relative 2^-24 |v - m|, doubled
for the sum's terms), expf's 2 ulp and a sum of E terms in log2(E) + E / 32
additions: relative error (2 span + 80) 2^-24 with span = max |v - m| over the terms
that count.  Gradient p_e (dw_e - dot): three such factors on p_e (|dw_e| + sum |p
dw|).  bf16 gradients: half a bf16 ulp more.  Values below 2^-126 may flush.
"""
import numpy as np
import pytest
import torch

from parity_bounds import bf16_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from fp4_weight_grouped_gb300 import binding
    binding.load()
    return binding


def reference(l, k, renorm):
    """float64 logits -> ids, softmax p over the experts that count (0 elsewhere)."""
    key = np.where(np.isnan(l), -np.inf, l)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    x = l
    if renorm:
        x = np.full_like(l, -np.inf)
        np.put_along_axis(x, ids, np.take_along_axis(l, ids, 1), 1)
    with np.errstate(invalid="ignore"):
        m = np.where(np.isnan(x), -np.inf, x).max(1, keepdims=True)
        e = np.where(x == -np.inf, 0.0, np.exp(x - m))
        s = e.sum(1, keepdims=True)
        p = np.where(s == 0, 0.0, e / np.where(s == 0, 1, s))
        span = np.where(np.isfinite(x) & np.isfinite(m), m - x, 0).max(1, keepdims=True)
    return ids, p, span


def gradient(p, ids, dw):
    full = np.zeros_like(p)
    np.put_along_axis(full, ids, dw, 1)
    dot = (p * full).sum(1, keepdims=True)
    return p * (full - dot), p * (np.abs(full) + (p * np.abs(full)).sum(1, keepdims=True))


def check(B, logits, k, renorm, dw=None):
    l = logits.double().cpu().numpy()
    ids, p, span = reference(l, k, renorm)
    got_ids, got_w = B.topk_gate(logits, k, renorm=renorm)
    np.testing.assert_array_equal(got_ids.cpu().numpy(), ids)
    w = np.take_along_axis(p, ids, 1)
    rel = (2 * span + 80) * 2.0 ** -24
    g = got_w.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(g), np.isnan(w))
    fine = ~np.isnan(w)
    assert np.all((np.abs(g - w) <= rel * w + 2.0 ** -126)[fine])
    if dw is None:
        return
    dl = B.topk_gate_backward(logits, got_ids, dw, renorm=renorm)
    assert dl.dtype == logits.dtype and dl.shape == logits.shape
    ref, mag = gradient(p, ids, dw.double().cpu().numpy())
    bound = 3 * rel * mag + 2.0 ** -120
    if logits.dtype == torch.bfloat16:
        bound = bound + bf16_ulp(ref) / 2
    d = dl.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(d), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.all((np.abs(d - ref) <= bound)[ok]), float((np.abs(d - ref) / bound)[ok].max())


CASES = [(1, 1, 1), (1, 2, 2), (5, 8, 2), (3, 31, 31), (7, 33, 4), (130, 64, 8), (64, 256, 6), (9, 257, 6), (17, 500, 5),
         (4, 1024, 8), (2, 1024, 1024), (1001, 100, 3)]


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", CASES)
def test_gate_and_gradient(B, T, E, k, dtype, renorm):
    g = torch.Generator(device=DEV).manual_seed(T * E + k)
    logits = (torch.randn((T, E), generator=g, device=DEV) * 2).to(dtype)
    check(B, logits, k, renorm, torch.randn((T, k), generator=g, device=DEV))


@pytest.mark.parametrize("renorm", [False, True])
def test_ties_zeros_and_masks(B, renorm):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    rows = [[1.0] * 40, [0.0, -0.0] * 20, [-inf] * 40, [-inf] * 39 + [2.0], [low] * 40, [low] * 20 + [-inf] * 20,
            [3.0, -inf] * 20, [nan] + [1.0] * 39, [-inf, nan] * 20, [nan] * 40, [inf] + [0.0] * 39, [88.0, -88.0] * 20,
            [1e30, -1e30] * 20]
    logits = torch.tensor(rows, device=DEV)
    for k in (1, 3, 40):
        check(B, logits, k, renorm, torch.ones((len(rows), k), device=DEV))


def test_row_strides(B):
    big = torch.randn((50, 300), device=DEV)
    for lo, hi in ((0, 256), (3, 67), (299, 300)):
        v = big[:, lo:hi]
        k = min(4, hi - lo)
        a, b = B.topk_gate(v, k), B.topk_gate(v.contiguous(), k)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        dw = torch.randn((50, k), device=DEV)
        assert torch.equal(B.topk_gate_backward(v, a[0], dw), B.topk_gate_backward(v.contiguous(), a[0], dw))
    one = torch.randn(64, device=DEV).expand(5, 64)        # row stride 0
    ids, _ = B.topk_gate(one, 3)
    assert torch.equal(ids, B.topk_gate(one.contiguous(), 3)[0])


def test_no_tokens_and_ids_out_of_range(B):
    ids, w = B.topk_gate(torch.zeros((0, 16), device=DEV), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert B.topk_gate_backward(torch.zeros((0, 16), device=DEV), ids, w).shape == (0, 16)
    logits = torch.randn((3, 16), device=DEV)
    dw = torch.randn((3, 3), device=DEV)
    bad = torch.tensor([[0, -1, 5], [16, 2, 2 ** 31 - 1], [1, 3, -2 ** 31]], dtype=torch.int32, device=DEV)
    keep = (bad >= 0) & (bad < 16)
    dl = B.topk_gate_backward(logits, bad, dw)
    safe = torch.where(keep, bad, 0)
    assert torch.allclose(dl, B.topk_gate_backward(logits, safe, torch.where(keep, dw, 0.0)), atol=1e-7)


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_formula_against_differences(renorm):
    """The formula that check() holds the kernel to, against central differences of
    the 64-bit weights (step 1e-5: truncation about 1e-10, rounding about 1e-11)."""
    rng = np.random.default_rng(0)
    l, dw = rng.standard_normal((4, 12)), rng.standard_normal((4, 3))
    ids, p, _ = reference(l, 3, renorm)
    ref, _ = gradient(p, ids, dw)

    def loss(x):      # the choice is held: it is piecewise constant
        x = np.take_along_axis(x, ids, 1) if renorm else x
        e = np.exp(x - x.max(1, keepdims=True))
        q = e / e.sum(1, keepdims=True)
        return ((q if renorm else np.take_along_axis(q, ids, 1)) * dw).sum(1)

    for e in range(12):
        step = np.zeros(12)
        step[e] = 1e-5
        np.testing.assert_allclose((loss(l + step) - loss(l - step)) / 2e-5, ref[:, e], atol=1e-8)


def test_refusals(B):
    x = torch.zeros((4, 16), device=DEV)
    for k in (0, 17):
        with pytest.raises(B.MoeError):
            B.topk_gate(x, k)
    with pytest.raises(B.MoeError):
        B.topk_gate(torch.zeros((1, 1025), device=DEV), 1)
    with pytest.raises(ValueError):
        B.topk_gate(x.half(), 2)
    with pytest.raises(ValueError):
        B.topk_gate(x.T, 2)
    ids, w = B.topk_gate(x, 2)
    with pytest.raises(ValueError):
        B.topk_gate_backward(x, ids.long(), w)
    with pytest.raises(ValueError):
        B.topk_gate_backward(x, ids, w[:, :1])
