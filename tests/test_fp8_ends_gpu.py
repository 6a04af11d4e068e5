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


# ---- products ---------------------------------------------------------------------
# every kind of tile: one nonzero code of 1.0 in each row of b picks an entry of
# a, so each result is one product
PICKS = [(5, 150, 300), (640, 730, 300), (1500, 1420, 700), (3100, 3300, 300), (4090, 3900, 129), (200, 300, 8192)]


def matrix(codes, scale_bytes):
    rows, cols = codes.shape
    q = mh().Fp8Matrix.empty(rows, cols)
    full = np.zeros(tuple(q.codes.shape), np.uint8)
    full[:, :cols] = codes
    q.codes.view(torch.uint8).copy_(torch.from_numpy(full))
    nb = -(-cols // 128)
    s = np.zeros(tuple(q.scales.shape), np.uint8)
    s[:, :nb] = scale_bytes
    q.scales.view(torch.uint8).copy_(torch.from_numpy(s))
    return q, fo.decode(codes) * np.ldexp(1.0, np.repeat(s[:, :nb].astype(np.int64), 128, axis=1)[:, :cols] - 127)


def picked(m, n, k, low, high, byte_b, limit, seed):
    """(a, b, exact results): a's scale bytes in [low, high], entries below
    `limit` in magnitude, b's all byte_b."""
    rng = np.random.default_rng((seed, m, n, k))
    nb = -(-k // 128)
    s = rng.integers(low, high + 1, (m, nb))
    codes = rng.integers(0, 127, (m, k)).astype(np.uint8)
    scale = np.ldexp(1.0, np.repeat(s, 128, axis=1)[:, :k] - 127)
    # codes whose entries would reach the limit lose 2^4 .. 2^8 of their exponent
    while np.any(bad := fo.decode(codes) * scale >= limit):
        codes = np.where(bad, codes - 8, codes).astype(np.uint8)
    codes |= (128 * rng.integers(0, 2, codes.shape)).astype(np.uint8)
    col = rng.integers(0, k, n)
    cb = np.zeros((n, k), np.uint8)
    cb[np.arange(n), col] = 56
    a, va = matrix(codes, s)
    b, _ = matrix(cb, np.full((n, nb), byte_b))
    return a, b, va[:, col] * 2.0 ** (byte_b - 127)


@pytest.mark.parametrize("dtype,fast", [("bf16", False), ("fp32", False), ("bf16", True)])
@pytest.mark.parametrize("m,n,k", PICKS)
def test_entries_at_the_ends_of_the_range(m, n, k, dtype, fast):
    """Up to the largest that fp32 holds, with scale bytes up to 254, entries
    count exactly, with bytes down to 0 to within half of bf16's smallest
    value, 2^-134; fast results take all entries exactly."""
    for low, high, byte_b in ((0, 20, 247), (226, 254, 20)):
        a, b, v = picked(m, n, k, low, high, byte_b, np.inf if fast else 2.0 ** 128, 51)
        out = mh().fp8_matmul(a, b, out_dtype=DT[dtype], fast=fast).double().cpu().numpy()
        if low and not fast or fast:
            assert np.array_equal(out, v)
        else:
            assert (np.abs(out - v) <= 2.0 ** -134 * 2.0 ** (byte_b - 127)).all()
            whole = v == np.round(v * 2.0 ** (133 - byte_b + 127)) * 2.0 ** (byte_b - 127 - 133)
            assert np.array_equal(out[whole], v[whole]) and 0.5 < whole.mean() < 1


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_an_entry_past_fp32_counts_as_infinite(dtype):
    """The largest fp32 values are coded 256 * 2^120."""
    x = torch.full((3, 128), 3.4e38, device="cuda")
    x[1] = 3.2e38
    x[2] = -3.4e38
    q, _ = mh().fp8_quantize(x)
    assert [int(v) for v in q.scales.view(torch.uint8)[:, 0]] == [247, 247, 247]
    w, _ = mh().fp8_quantize(torch.full((5, 128), 2.0 ** -60, device="cuda"))
    out = mh().fp8_matmul(q, w, out_dtype=DT[dtype])
    assert (out[0] == float("inf")).all() and (out[2] == -float("inf")).all()
    assert (out[1] == 128 * 240 * 2.0 ** 60).all()  # 3.2e38 = 240.7 * 2^120
    assert torch.equal(q.dequantize()[0], torch.full((128,), float("inf"), device="cuda"))


@pytest.mark.parametrize("dtype,fast", [("bf16", False), ("fp32", False), ("bf16", True)])
def test_the_scale_byte_255_is_nan(dtype, fast):
    a, _ = matrix(np.full((4, 300), 56, np.uint8), np.full((4, 3), 127))
    a.scales.view(torch.uint8)[2, 1] = 255
    b, _ = matrix(np.full((7, 300), 56, np.uint8), np.full((7, 3), 127))
    out = mh().fp8_matmul(a, b, out_dtype=DT[dtype], fast=fast)
    assert torch.isnan(out[2]).all() and (out[[0, 1, 3]] == 300.0).all()
