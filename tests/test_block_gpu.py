"""The operators together, as a training step uses them: token ids -> embedding -> norm
with an 8-bit (or 4-bit) output -> a linear layer -> gradients back to the table -> MuonH for
the matrix, AdamW for the table and the norm's weight.

Each result is compared with an fp64 computation from the tensors that went into its
operator (the quantized operands' values among them), so that bounds stay those of
single operators: u = 2^-24; bf16 results half a step, 2^-8; fp32 sums of k terms (k + 64) u
of the sum of magnitudes."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import adamw_step

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
VOCAB, D, N, SHAPE = 700, 384, 520, (2, 150)


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def mh():
    import orthogonalized_updates_amd
    return orthogonalized_updates_amd


def near(got, want, terms, size, half):
    """got: a result; want, size: the exact value and the sum of its terms' magnitudes."""
    err = (got.double() - want).abs()
    return bool((err <= terms * U * size + half * want.abs() + 1e-44).all())


class Model:
    def __init__(self, bits):
        m = mh()
        g = torch.Generator(device="cuda").manual_seed(3)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.bits = bits
        self.table, self.scale = r(VOCAB, D) * 0.02, math.sqrt(D)
        self.w = 1 + 0.1 * r(D)
        self.stream = r(*SHAPE, D).bfloat16()       # another part's share of the residual stream
        self.W, self.M = [r(N, D) * 0.05], [torch.zeros(N, D, device="cuda")]
        self.opt = m.MuonH([(N, D)])
        self.opt.init(self.W)
        self.set8 = self.opt.quantize_weights(self.W, self.opt.fp8_weights())
        self.rest = m.AdamW([VOCAB * D, D])
        self.state = [torch.zeros_like(t) for t in (self.table, self.w) for _ in range(2)]
        # ids with repetitions and padding
        self.ids = torch.randint(0, VOCAB, SHAPE, device="cuda", generator=g)
        self.ids[:, ::3] = 7
        self.ids[1, -20:] = -1
        self.dy = (r(SHAPE[0] * SHAPE[1], N) * 1e-3).bfloat16()
        self.dstream = (r(SHAPE[0] * SHAPE[1], D) * 1e-3).bfloat16()
        self.G, self.dtable, self.dw = torch.empty(N, D, device="cuda"), torch.empty(VOCAB, D, device="cuda"), torch.empty(D, device="cuda")

    def forward_backward(self):
        m = mh()
        x = m.embedding(self.ids, self.table, scale=self.scale, out_dtype=torch.bfloat16)
        flat, stream = x.view(-1, D), self.stream.view(-1, D)
        if self.bits == 8:
            q, qt, h, r = m.rms_norm_fp8(flat, self.w, residual=stream, forms="both")
            w, wt, mul = self.set8.weights[0], self.set8.transposed[0], m.fp8_matmul
            d, dt = m.fp8_quantize(self.dy, forms="both")
        else:
            y, h, r = m.rms_norm(flat, self.w, residual=stream)
            q, qt = m.fp4_quantize(y, forms="both")
            w, wt = m.fp4_quantize(self.W[0], forms="both")
            d, dt = m.fp4_quantize(self.dy, forms="both")
            mul = m.fp4_matmul
        y = mul(q, w)
        dn = mul(d, wt)
        mul(dt, qt, out=self.G)
        dh, dw = m.rms_norm_backward(dn, h, self.w, r, dresidual=self.dstream, dweight=self.dw)
        m.embedding_backward(self.ids, dh.view(*SHAPE, D), self.dtable, scale=self.scale)
        return dict(x=x, q=q, qt=qt, h=h, r=r, w=w, wt=wt, d=d, dt=dt, y=y, dn=dn, dh=dh)

    def update(self, step):
        self.opt.step(self.W, [self.G], self.M, lr=0.02, fp8=self.set8)
        self.rest.step([self.table, self.w], [self.dtable, self.dw], self.state[0::2], self.state[1::2], lr=1e-3, step=step)


@pytest.mark.parametrize("bits", [8, 4])
def test_training_steps(bits):
    t = Model(bits)
    keep = t.ids.view(-1) >= 0
    for step in (1, 2):
        got = t.forward_backward()
        v = {k: got[k].dequantize().double() for k in ("q", "qt", "w", "wt", "d", "dt")}
        # forward
        want = t.table.double()[t.ids.clamp_min(0)] * t.scale * (t.ids >= 0)[..., None]
        assert near(got["x"], want, 2, want.abs(), 2.0 ** -8)
        h = (got["x"].float() + t.stream.float()).bfloat16().view(-1, D)
        assert torch.equal(got["h"], h)
        r = 1 / (h.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
        norm = h.double() * r * t.w.double()
        # half a step of the format beside the largest entry of a block: at most 1 of more than 4 (4 bits, and
        # bf16's 2^-8 before), 16 of more than 256 (8 bits)
        top = norm.abs().max()
        for p, n in ((v["q"], norm), (v["qt"], norm.t())):
            assert float((p - n).abs().max()) <= float(top) * (1 / 4 + 2.0 ** -7 if bits == 4 else 1 / 16 + 2.0 ** -20)
        assert near(got["y"], v["q"] @ v["w"].t(), 8 * 3 + 64, v["q"].abs() @ v["w"].abs().t(), 2.0 ** -8)
        # backward
        assert near(got["dn"], v["d"] @ v["wt"].t(), 8 * 5 + 64, v["d"].abs() @ v["wt"].abs().t(), 2.0 ** -8)
        assert near(t.G, v["dt"] @ v["qt"].t(), 8 * 3 + 64, v["dt"].abs() @ v["qt"].abs().t(), U)
        n, dn = h.double() * r, got["dn"].double()
        g = dn * t.w.double()
        mean = (g * n).mean(1, keepdim=True)
        dh = r * (g - n * mean) + t.dstream.double()
        size = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) + t.dstream.double().abs()
        assert near(got["dh"], dh, 64, size, 2.0 ** -8)
        assert near(t.dw, (dn * n).sum(0), 128, (dn * n).abs().sum(0), U)
        grads = got["dh"].double()[keep] * t.scale
        want = torch.zeros(VOCAB, D, dtype=torch.float64, device="cuda").index_add_(0, t.ids.view(-1)[keep], grads)
        assert near(t.dtable, want, 200, torch.zeros_like(want).index_add_(0, t.ids.view(-1)[keep], grads.abs()), U)
        # updates: every row of the table (weight decay reaches those without a token too)
        before = [x.clone() for x in (t.table, t.w, *t.state)]
        W = t.W[0].clone()
        t.update(step)
        for i, (p, grad) in enumerate(((t.table, t.dtable), (t.w, t.dw))):
            ref = adamw_step(before[i].cpu().numpy(), grad.cpu().numpy(), before[2 + 2 * i].cpu().numpy(), before[3 + 2 * i].cpu().numpy(), 1e-3, 0.9, 0.95,
                             1e-8, 0.1, step)
            assert np.allclose(p.cpu().numpy(), ref[0], rtol=1e-5, atol=1e-7)
        assert not torch.equal(W, t.W[0]) and t.opt.status() == 0
        assert torch.equal(t.set8.weights[0].dequantize(), mh().fp8_quantize(t.W[0], block="tiles")[0].dequantize())


@pytest.mark.parametrize("bits", [8, 4])
def test_a_captured_step_replays(bits):
    t = Model(bits)
    t.forward_backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = t.forward_backward()
    for i in range(3):
        t.ids.copy_(torch.randint(-1, VOCAB, SHAPE, device="cuda"))
        t.dy.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [held["y"].clone(), held["dh"].clone(), t.G.clone(), t.dtable.clone(), t.dw.clone()]
        again = t.forward_backward()
        assert all(torch.equal(a, b) for a, b in zip(got, [again["y"], again["dh"], t.G, t.dtable, t.dw]))
        t.update(i + 1)  # the captured step reads what the optimizers changed in place


def test_one_token():
    """The serving form: a single token through embedding, norm and both kinds of linear layer."""
    t = Model(8)
    m = mh()
    one = torch.tensor([3], device="cuda")
    x = m.embedding(one, t.table, scale=t.scale, out_dtype=torch.bfloat16)
    q, _, h, r = m.rms_norm_fp8(x, t.w, residual=t.stream.view(-1, D)[:1])
    y = m.fp8_matmul(q, t.set8.weights[0])
    assert near(y, q.dequantize().double() @ t.set8.weights[0].dequantize().double().t(), 128,
                q.dequantize().double().abs() @ t.set8.weights[0].dequantize().double().abs().t(), 2.0 ** -8)
    w4 = m.fp4_quantize(t.W[0])[0]
    n = m.rms_norm(x, t.w, residual=t.stream.view(-1, D)[:1])[0]
    q4 = m.fp4_quantize(n)[0]
    y4 = m.fp4_matmul(q4, w4)
    assert near(y4, q4.dequantize().double() @ w4.dequantize().double().t(), 128,
                q4.dequantize().double().abs() @ w4.dequantize().double().abs().t(), 2.0 ** -8)
