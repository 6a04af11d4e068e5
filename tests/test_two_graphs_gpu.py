"""Calls that take a workspace, in two captured graphs: replayed in turn with eager
calls between them, and on two streams at once, bit for bit the eager results. Each
call's workspace is its own."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def mh():
    import orthogonalized_updates_amd
    return orthogonalized_updates_amd


def inputs(kind, seed):
    """A function of an output tensor that makes a call, and that output's shape."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    m = mh()
    if kind.startswith("embedding"):
        n = int(kind.split()[1])
        ids = torch.randint(-5, 400, (n,), device="cuda", generator=g)
        ids[: n // 2] = 3  # a row whose sum is shared out
        dy = r(n, 600).bfloat16()
        return lambda out: m.embedding_backward(ids, dy, out), (400, 600)
    if kind == "norm":
        x, dy, w = r(3000, 1000), r(3000, 1000), 1 + 0.1 * r(1000)
        rstd = m.rms_norm(x, w)[2]
        return lambda out: m.rms_norm_backward(dy, x, w, rstd, dweight=out), (1000,)
    a, b = m.fp4_quantize(r(200, 16384))[0], m.fp4_quantize(r(300, 16384))[0]
    assert m.get_lib().muonh_fp4_matmul_workspace_bytes(200, 300, 16384) > 0
    return lambda out: m.fp4_matmul(a, b, out=out), (200, 300)


@pytest.mark.parametrize("kind", ["embedding 500", "embedding 5000", "embedding 30000", "norm", "product"])
def test_two_captured_graphs(kind):
    calls, shapes = zip(*[inputs(kind, 40 + i) for i in range(3)])
    want = [torch.empty(s, device="cuda") for s in shapes]
    for call, w in zip(calls, want):
        call(w)
    outs = [torch.empty(s, device="cuda") for s in shapes]
    torch.cuda.synchronize()
    graphs = []
    for call, out in zip(calls[:2], outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out)
        graphs.append(graph)
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            out.fill_(float("nan"))
            graph.replay()
            calls[2](outs[2])
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            calls[2](outs[2])
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
