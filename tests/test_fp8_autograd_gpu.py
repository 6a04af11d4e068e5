"""The 8-bit operators inside a torch.autograd.Function on the GPU, and the
versions of what they write into."""
from __future__ import annotations

import numpy as np
import pytest

from test_fp8_gpu import bound, host, mh, need_gpu  # noqa: F401
from oracle import fp8_oracle as fo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_versions_of_given_outputs_move():
    m = mh()
    x = torch.randn(130, 200, device="cuda", requires_grad=True)
    q, qt = m.fp8_quantize(x, forms="both")
    assert not q.codes.requires_grad
    for t in (q.codes, q.scales, qt.codes, qt.scales):
        assert t._version == 0
    m.fp8_quantize(x, forms="both", out=q, out_t=qt)
    for t in (q.codes, q.scales, qt.codes, qt.scales):
        assert t._version == 1
    out = torch.zeros(130, 130, device="cuda")
    m.fp8_matmul(q, q, out=out, accumulate=True)
    assert out._version == 1
    opt = m.MuonH([(64, 64)])
    ws = opt.fp8_weights()
    v = ws.weights[0].codes._version
    opt.quantize_weights([torch.randn(64, 64, device="cuda")], ws)
    assert ws.weights[0].codes._version == v + 1 and ws.transposed[0].scales._version == ws.storage._version


def test_a_linear_layer_in_a_function():
    """Y = X W^T with its gradients as a Function's forward and backward, in a
    graph of other operations: the gradients of the formula on quantized
    values, to the products' bounds."""
    m = mh()
    t, n, k = 150, 260, 200

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            qx, qxt = m.fp8_quantize(x, forms="both")
            qw, qwt = m.fp8_quantize(w, block="tiles", forms="both")
            ctx.saved = qxt, qwt
            return m.fp8_matmul(qx, qw, out_dtype=torch.float32)

        @staticmethod
        def backward(ctx, dy):
            qxt, qwt = ctx.saved
            qd, qdt = m.fp8_quantize(dy.contiguous(), forms="both")
            return m.fp8_matmul(qd, qwt, out_dtype=torch.float32), m.fp8_matmul(qdt, qxt, out_dtype=torch.float32)

    g = torch.Generator("cuda").manual_seed(12)
    x = torch.randn(t, k, device="cuda", generator=g).requires_grad_()
    w = (torch.randn(n, k, device="cuda", generator=g) * 0.05).requires_grad_()
    c = torch.randn(t, n, device="cuda", generator=g)
    y = Linear.apply(x, w)
    (2 * y * c).sum().backward()
    vals = lambda z, **kw: [fo.values(*host(q), q.shape, q.block) for q in m.fp8_quantize(z, forms="both", **kw)]  # noqa: E731
    with torch.no_grad():
        vx, vxt = vals(x)
        vw, vwt = vals(w, block="tiles")
        vd, vdt = vals(2 * c)  # exactly what reaches the backward pass
    for got, a, b in ((y, vx, vw), (x.grad, vd, vwt), (w.grad, vdt, vxt)):
        v, tol = bound(a, b, a @ b.T, "fp32")
        assert (np.abs(got.detach().double().cpu().numpy() - v) <= tol).all()
