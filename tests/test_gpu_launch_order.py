"""Calls right behind whatever writes their inputs, eager and captured: a kernel, a copy from the
host, a memset, work of another stream joined by an event, another call of the library.  Launches
within a call may start under the end of one another, and must read nothing too early."""
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


@pytest.fixture(scope="module")
def data(B):
    g = torch.Generator(device="cuda").manual_seed(4)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    d = dict(codes=torch.randint(0, 256, (64, 512, 256), generator=g, device="cuda", dtype=torch.uint8),
             scales=torch.randint(115, 125, (64, 512, 16), generator=g, device="cuda", dtype=torch.uint8),
             src=bf(40, 512), ids=torch.randint(0, 64, (40,), generator=g, device="cuda", dtype=torch.int32),
             w13=bf(256, 512), w2=bf(512, 128), big=torch.randn(1 << 26, generator=g, device="cuda"),
             ws=torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"))
    d["host"], d["host_ids"] = d["src"].cpu().pin_memory(), d["ids"].cpu().pin_memory()
    torch.cuda.synchronize()
    return d


def calls(B, d, x, ids):
    """A product, the block forward and backward, and clipping of its gradients, each behind the other."""
    ws = d["ws"]
    y = B.fp4_matvec(x, d["codes"], d["scales"], 0, row_expert=ids, workspace=ws)
    h, gu = x.new_empty((40, 128)), x.new_empty((40, 256))
    out = B.ffn_forward(x, d["w13"], d["w2"], h=h, gu=gu, workspace=ws)
    grads = list(B.ffn_backward(out, x, d["w13"], d["w2"], h, gu, workspace=ws))
    norm = B.clip_grads(grads, 0.5, workspace=ws)
    one = B.fp4_matvec(grads[0][:2], d["codes"], d["scales"], 0, row_expert=ids[:2], workspace=ws)
    return [y, out, norm, one] + grads


def writers(d, x, ids):
    other = torch.cuda.Stream()

    def kernel():
        d["big"].mul_(1.0)
        x.copy_(d["src"])
        ids.copy_(d["ids"])

    def host():
        x.copy_(d["host"], non_blocking=True)
        ids.copy_(d["host_ids"], non_blocking=True)

    def memset():
        x.copy_(d["src"])
        ids.copy_(d["ids"])
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").zero_()

    def joined():
        here = torch.cuda.current_stream()
        start, end = torch.cuda.Event(), torch.cuda.Event()
        start.record(here)
        with torch.cuda.stream(other):
            other.wait_event(start)
            d["big"].mul_(1.0)
            x[:20].copy_(d["src"][:20])
            ids.copy_(d["ids"])
            end.record(other)
        x[20:].copy_(d["src"][20:])
        here.wait_event(end)

    return dict(kernel=kernel, host=host, memset=memset, joined=joined)


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("writer", ["kernel", "host", "memset", "joined"])
def test_behind(B, data, writer, captured):
    x, ids = data["src"].clone(), data["ids"].clone()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        want = [t.clone() for t in calls(B, data, x, ids)]
        stream.synchronize()
        write = writers(data, x, ids)[writer]
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                write()
                got = calls(B, data, x, ids)
        for _ in range(5):
            x.fill_(7.0)
            ids.fill_(3)
            stream.synchronize()
            if captured:
                graph.replay()
            else:
                write()
                got = calls(B, data, x, ids)
            stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), writer


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "graph"])
def test_behind_a_grouped_product_of_both_band_classes(B, captured):
    """The grouped product's two launches run beside each other; a call behind them sees the rows of
    both.  Many short bands (the first launch's) and one of 40 rows."""
    g = torch.Generator(device="cuda").manual_seed(9)
    E, N, K = 128, 512, 4096
    sizes = torch.full((E,), 31, dtype=torch.int32)
    sizes[0] = 40
    rows, sizes = int(sizes.sum()), sizes.cuda()
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(115, 122, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    act = torch.randn((rows, K), generator=g, device="cuda").bfloat16()
    w13 = torch.randn((256, N), generator=g, device="cuda").bfloat16()
    w2 = torch.randn((N, 128), generator=g, device="cuda").bfloat16()
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    ids = torch.arange(64, device="cuda", dtype=torch.int32)
    c2 = torch.randint(0, 256, (64, 64, N // 2), generator=g, device="cuda", dtype=torch.uint8)
    s2 = torch.randint(115, 122, (64, 64, N // 32), generator=g, device="cuda", dtype=torch.uint8)

    def run():
        B.grouped_gemm(act, codes, scales, sizes, out=y, workspace=ws)
        few = B.fp4_matvec(y[-64:], c2, s2, 0, row_expert=ids, workspace=ws)
        B.grouped_gemm(act, codes, scales, sizes, out=y, workspace=ws)
        return few, B.ffn_forward(y, w13, w2, workspace=ws)

    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    if captured:
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = run()
    for _ in range(10):
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
