"""Block-scaled 8-bit operators at both ends of the range, on the GPU: whole
blocks of the lowest scale 2^-126 (subnormal sources among them, where every
code takes a rounding decision) and entries next to the largest fp32 value."""
from __future__ import annotations

import numpy as np
import pytest

from test_fp8_gpu import DT, check_matrix, mh, need_gpu  # noqa: F401
from oracle import fp8_oracle as fo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def bottom(rows, cols, kind, seed):
    """fp32 values whose blocks have scale 2^-126 or one near it."""
    rng = np.random.default_rng((seed, rows, cols))
    g = fo.grid()
    if kind == "bits":  # any bit pattern up to 448 * 2^-126, and a row's own limit
        top = int(np.float32(448 * 2.0 ** -126).view(np.uint32))
        limit = np.exp2(rng.uniform(0, np.log2(top), (rows, 1))).astype(np.int64)
        bits = (rng.random((rows, cols)) * (limit + 1)).astype(np.uint32)
        x = bits.view(np.float32).astype(np.float64)
    elif kind == "halfway":  # codes and points halfway between two, at scale 2^-126
        pool = np.concatenate([g, (g[1:] + g[:-1]) / 2])
        x = rng.choice(pool, (rows, cols)) * 2.0 ** -126
    elif kind == "beside":  # the neighbours of the halfway points, where fp32 has them
        mid = ((g[1:] + g[:-1]) / 2 * 2.0 ** -126).astype(np.float32)
        pool = np.concatenate([np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1))])
        x = rng.choice(pool, (rows, cols)).astype(np.float64)
    else:  # both sides of the lowest scale: a block's largest entry at 448 * 2^-126 and the next floats
        edge = np.float32(448 * 2.0 ** -126)
        peaks = np.array([np.nextafter(edge, np.float32(0)), edge, np.nextafter(edge, np.float32(1)),
                          np.float32(449 * 2.0 ** -126), np.float32(2.0 ** -126), np.float32(2.0 ** -149)], np.float64)
        x = rng.random((rows, cols)) * 2.0 ** -126
        peak = rng.choice(peaks, (rows, -(-cols // 128)))
        x = np.minimum(x, np.repeat(peak, 128, axis=1)[:, :cols])
        x[:, ::128] = peak
    return (x * rng.choice([-1.0, 1.0], (rows, cols))).astype(np.float32)


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["bits", "halfway", "beside", "edge"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (130, 300), (257, 129)])
def test_quantize_at_the_lowest_scale(rows, cols, kind, dtype, block):
    x = torch.from_numpy(bottom(rows, cols, kind, 1)).to(DT[dtype])
    x64 = x.double().numpy()  # on the host, which keeps subnormal values
    q, qt = mh().fp8_quantize(x.cuda(), block=block, forms="both")
    check_matrix(q, x64, block)
    check_matrix(qt, x64.T, block)
    for forms, ref in (("plain", q), ("transposed", qt)):
        one = next(o for o in mh().fp8_quantize(x.cuda(), block=block, forms=forms) if o is not None)
        assert torch.equal(one.codes.view(torch.uint8), ref.codes.view(torch.uint8))
        assert torch.equal(one.scales.view(torch.uint8), ref.scales.view(torch.uint8))


def test_the_inputs_round_at_the_lowest_scale():
    """What the test above stands on: most entries lie in blocks of the lowest
    scale, are nonzero, and most of those of some kinds are no code's value."""
    for kind in ("bits", "halfway", "beside", "edge"):
        x = bottom(130, 300, kind, 1).astype(np.float64)
        codes, scales = fo.quantize(x)
        low = np.repeat(scales[:, :3] == 1, 128, axis=1)[:, :300] & (x != 0)
        assert low.mean() > 0.3
        inexact = fo.values(codes, scales, x.shape) != x
        if kind != "edge":
            assert (low & inexact).mean() > 0.3


def test_weights_at_the_lowest_scale():
    shapes = [(130, 300), (257, 129)]
    W = [torch.from_numpy(bottom(*s, "bits", 2)) for s in shapes]
    opt = mh().MuonH(shapes)
    ws = opt.quantize_weights([w.cuda() for w in W], opt.fp8_weights())
    for w, q, qt in zip(W, ws.weights, ws.transposed):
        check_matrix(q, w.double().numpy(), "tiles")
        check_matrix(qt, w.double().numpy().T, "tiles")
