"""Block-scaled products whose blocks of k are split over workgroups (few
output tiles, long sums; a second launch joins the partial sums), on the GPU
against fp64: what test_fp8_gpu.py and test_fp8_sums_gpu.py ask of products at
other sizes, with the bounds given there."""
from __future__ import annotations

import numpy as np
import pytest

from test_fp8_gpu import DT, check_product, host, mh, need_gpu, operand  # noqa: F401
from test_fp8_sums_gpu import HALF_STEP, cancelling, spread
from oracle import fp8_oracle as fo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ab", [("rows", "rows"), ("tiles", "tiles")])
@pytest.mark.parametrize("extra,first", [(0, 0), (53, 0), (0, 1), (61, 8)])
@pytest.mark.parametrize("m,n,k", [(200, 301, 8192), (140, 150, 9000), (20, 2000, 6001)])
def test_split_products_add_into_strided_rows(m, n, k, extra, first, ab, dtype):
    ld = n + extra
    a, va = operand(m, k, 41, ab[0], spread=False)
    b, vb = operand(n, k, 42, ab[1], spread=False)
    buf = torch.full((m * ld + 64,), 7.0, dtype=DT[dtype], device="cuda")
    out = buf[first:first + (m - 1) * ld + n].as_strided((m, n), (ld, 1), first)
    for acc in (False, True, False):
        old = out.double().cpu().numpy() if acc else None
        mh().fp8_matmul(a, b, out=out, accumulate=acc)
        check_product(out, va, vb, dtype, old)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[first:first + (m - 1) * ld + n].as_strided((m, n), (ld, 1), first).fill_(False)
    assert (buf[mask] == 7.0).all()
    assert torch.equal(mh().fp8_matmul(a, b, out_dtype=DT[dtype]), out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", [(200, 300, 8192), (300, 260, 9000)])
def test_split_sums_are_fp32(m, n, k, dtype):
    (a, va), (b, vb) = cancelling(m, n, k, 43)
    v, p = va @ vb.T, np.abs(va) @ np.abs(vb).T
    sums = (k / 32 + 64) * 2.0 ** -24 * p
    err = np.abs(mh().fp8_matmul(a, b, out_dtype=DT[dtype]).double().cpu().numpy() - v)
    assert (err <= HALF_STEP[dtype] * np.abs(v) + sums).all()


@pytest.mark.parametrize("m,n,k", [(200, 300, 8192), (150, 203, 6000), (20, 2000, 6001)])
def test_split_fast_results_keep_their_bound(m, n, k):
    (a, va), (b, vb) = spread(m, k, 44), spread(n, k, 45)
    v, p = va @ vb.T, np.abs(va) @ np.abs(vb).T
    tol = 15 * 2.0 ** -13 * p + (k / 16 + 64) * 2.0 ** -24 * p
    err = np.abs(mh().fp8_matmul(a, b, fast=True).double().cpu().numpy() - v)
    assert (err <= tol + 2.0 ** -8 * (np.abs(v) + tol)).all()


@pytest.mark.parametrize("dtype,fast", [("bf16", False), ("bf16", True), ("fp32", False)])
@pytest.mark.parametrize("m,n,k", [(200, 300, 8192)])
def test_split_products_keep_nan_in_its_rows(m, n, k, dtype, fast):
    g = torch.Generator("cuda").manual_seed(46)
    x, w = torch.randn(m, k, device="cuda", generator=g), torch.randn(n, k, device="cuda", generator=g)
    x[2, 7] = float("nan")
    x[130, 8100] = float("inf")
    w[9, 4000] = -float("inf")
    a, b = mh().fp8_quantize(x)[0], mh().fp8_quantize(w)[0]
    out = mh().fp8_matmul(a, b, out_dtype=DT[dtype], fast=fast).double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        v = fo.values(*host(a), (m, k)) @ fo.values(*host(b), (n, k)).T
    assert np.array_equal(np.isnan(out), np.isnan(v)) and np.isfinite(out[~np.isnan(v)]).all()
    assert np.isnan(v).sum() == 2 * n + m - 2


def test_two_captured_graphs_keep_their_workspaces_apart():
    """A split product's partial sums live in a workspace of the call's own:
    two graphs with one each, replayed in turn and on two streams at once with
    eager products between them, all bit for bit the eager results."""
    m, n, k = 200, 300, 8192
    ops = [(operand(m, k, 50 + i, spread=False)[0], operand(n, k, 60 + i, spread=False)[0]) for i in range(3)]
    want = [mh().fp8_matmul(a, b, out_dtype=torch.float32) for a, b in ops]
    outs = [torch.zeros(m, n, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for (a, b), out in zip(ops, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mh().fp8_matmul(a, b, out=out)
            mh().fp8_matmul(a, b, out=out, accumulate=True)
        graphs.append(graph)
    twice = []
    for (a, b), w in zip(ops, want):
        twice.append(mh().fp8_matmul(a, b, out=w.clone(), accumulate=True))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            out.fill_(float("nan"))
            graph.replay()
            assert torch.equal(mh().fp8_matmul(*ops[2], out_dtype=torch.float32), want[2])
        torch.cuda.synchronize()
        assert all(torch.equal(out, t) for out, t in zip(outs, twice))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        assert torch.equal(mh().fp8_matmul(*ops[2], out_dtype=torch.float32), want[2])
        torch.cuda.synchronize()
        assert all(torch.equal(out, t) for out, t in zip(outs, twice))
