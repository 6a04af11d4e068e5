"""Block-scaled 8-bit operators on the GPU against the fp64 oracle.

Quantization is defined bit for bit: codes, scales and padding must be equal.

Products, element by element, with v the exact value and P = sum_k |a_k b_k|:
  bf16: the result's rounding, 2^-8 |v| (half a step), plus what the 8-bit
        matrix instructions drop: in a group of at most 16 products added at
        once, 15 lose at most 2^-13 of the largest each: 15 * 2^-13 P < 2^-9 P
        (fp32 sums come on top, far below that);
  fp32: its rounding, 2^-24 |v|, plus fp32 sums of exact products: k/32 + 64
        roundings in a row at most (32 inside an instruction, one per
        instruction, up to 16 partial sums, up to 8 waves' sums, the old
        value), (k/32 + 64) * 2^-24 P.
With accumulate, P and the bound count the old value too.
"""
from __future__ import annotations

import sys

import numpy as np
import pytest

from oracle import fp8_oracle as fo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def mh():
    import orthogonalized_updates_amd
    return orthogonalized_updates_amd


DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def values(rows, cols, seed, dtype="fp32"):
    """Sizes over many orders of magnitude between blocks, normal inside."""
    rng = np.random.default_rng((seed, rows, cols))
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    x *= np.exp2(rng.integers(-6, 7, (1, cols)))
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()


def special(rows, cols, seed, dtype):
    """NaN, infinities, zero blocks, halfway values, full-scale and tiny ones."""
    x = values(rows, cols, seed, dtype)
    rng = np.random.default_rng(seed)
    g = fo.grid()
    pool = np.concatenate([g, (g[1:] + g[:-1]) / 2, -g, [448, 448 * 2.0 ** 7, 450 * 2.0 ** -20, 2.0 ** -126,
                           2.0 ** -133, 3.3e38, np.inf, -np.inf, np.nan, -0.0, 0.0]])
    hit = torch.from_numpy(rng.random((rows, cols)) < 0.3).cuda()
    put = torch.from_numpy(rng.choice(pool, (rows, cols)).astype(np.float32)).to(x.dtype).cuda()
    x = torch.where(hit, put, x)
    x[:: 3, : 128] = 0.0
    if rows > 2 and cols > 130:
        x[1, 128:] = float("nan")
    return x


def host(m):
    return m.codes.view(torch.uint8).cpu().numpy(), m.scales.view(torch.uint8).cpu().numpy()


def same_codes(got, want):
    """Equal, except that any NaN code stands for NaN."""
    nan = (want & 127) == 127
    return np.array_equal(got[~nan], want[~nan]) and bool(((got[nan] & 127) == 127).all())


def check_matrix(m, x64, block):
    codes, scales = host(m)
    want_c, want_s = fo.quantize(x64, block)
    assert codes.shape == want_c.shape and scales.shape == want_s.shape
    assert np.array_equal(scales, want_s)
    assert same_codes(codes, want_c)


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (2048, 1), (3, 640), (127, 129), (128, 128), (129, 300),
                                       (257, 1001), (1000, 64), (640, 520)])
def test_quantize_is_the_definition(rows, cols, dtype, block):
    for x in (values(rows, cols, 5, dtype), special(rows, cols, 6, dtype)):
        q, qt = mh().fp8_quantize(x, block=block, forms="both")
        x64 = x.double().cpu().numpy()
        check_matrix(q, x64, block)
        check_matrix(qt, x64.T, block)
        for forms in ("plain", "transposed"):
            one = mh().fp8_quantize(x, block=block, forms=forms)
            assert [o is None for o in one] == [forms == "transposed", forms == "plain"]
            for o, ref in zip(one, (q, qt)):
                if o is not None:
                    assert torch.equal(o.codes.view(torch.uint8), ref.codes.view(torch.uint8))
                    assert torch.equal(o.scales.view(torch.uint8), ref.scales.view(torch.uint8))


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_quantize_of_every_kind_of_nan(dtype, block):
    """Quiet and signaling NaNs of either sign anywhere: NaN codes, and the
    largest finite entry still counts, whatever stands before or after it."""
    kinds = [0x7f800001, 0x7fbfffff, 0x7fc00000, 0x7fffffff] if dtype == "fp32" else [0x7f81, 0x7fbf, 0x7fc0, 0x7fff]
    sign, idt = (1 << 31, torch.int32) if dtype == "fp32" else (1 << 15, torch.int16)
    rng = np.random.default_rng(31)
    x = values(200, 264, 9, dtype)
    bits = x.view(idt).cpu().numpy()
    pick = rng.choice(np.array(kinds + [k | sign for k in kinds], np.uint64), bits.shape)
    hit = rng.random(bits.shape) < rng.choice([0.01, 0.2, 0.6], (200, 1))
    bits = np.where(hit, pick, bits.view(np.uint32 if dtype == "fp32" else np.uint16)).astype(
        np.uint32 if dtype == "fp32" else np.uint16)
    x = torch.from_numpy(bits.view(np.int32 if dtype == "fp32" else np.int16)).cuda().view(DT[dtype])
    x64 = np.where(hit, np.nan, values(200, 264, 9, dtype).double().cpu().numpy())
    q, qt = mh().fp8_quantize(x, block=block, forms="both")
    check_matrix(q, x64, block)
    check_matrix(qt, x64.T, block)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("ld,first", [(512, 0), (520, 8), (303, 0), (301, 1), (1024, 3)])
def test_quantize_of_strided_rows(ld, first, dtype):
    base = values(200, ld + 8, 7, dtype)
    x = base.reshape(-1)[first:first + 199 * ld + 300].as_strided((199, 300), (ld, 1))
    q, qt = mh().fp8_quantize(x, forms="both")
    check_matrix(q, x.double().cpu().numpy(), "rows")
    check_matrix(qt, x.double().cpu().numpy().T, "rows")


def guarded(rows, cols, block):
    """An Fp8Matrix inside larger buffers of a known byte, and those buffers."""
    m = mh()
    (r, ld), (sr, sld) = m._fp8_layout(rows, cols, block)
    bufs = [torch.full((r * ld + 512,), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((sr * sld + 512,), 0xA5, dtype=torch.uint8, device="cuda")]
    codes = bufs[0][256:256 + r * ld].view(torch.float8_e4m3fn).view(r, ld)
    scales = bufs[1][256:256 + sr * sld].view(torch.float8_e8m0fnu).view(sr, sld)
    return m.Fp8Matrix(codes, scales, (rows, cols), block), bufs


@pytest.mark.parametrize("block", ["rows", "tiles"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (130, 200), (257, 513)])
def test_quantize_writes_its_outputs_only(rows, cols, block):
    x = values(rows, cols, 8)
    q, bq = guarded(rows, cols, block)
    t, bt = guarded(cols, rows, block)
    mh().fp8_quantize(x, block=block, forms="both", out=q, out_t=t)
    check_matrix(q, x.double().cpu().numpy(), block)
    check_matrix(t, x.double().cpu().numpy().T, block)
    for b in bq + bt:
        assert (b[:256] == 0xA5).all() and (b[-256:] == 0xA5).all()


def test_quantize_of_nothing():
    for shape in ((0, 100), (100, 0), (0, 0)):
        q, qt = mh().fp8_quantize(torch.empty(shape, device="cuda"), forms="both")
        assert q.shape == shape and qt.shape == shape[::-1]


# ---- products --------------------------------------------------------------------
def operand(rows, cols, seed, block="rows", spread=True):
    """(Fp8Matrix, its fp64 values)."""
    x = values(rows, cols, seed) if spread else \
        torch.from_numpy(np.random.default_rng(seed).standard_normal((rows, cols)).astype(np.float32)).cuda()
    q, _ = mh().fp8_quantize(x, block=block)
    return q, fo.values(*host(q), (rows, cols), block)


def bound(va, vb, v, dtype, old=None):
    """(exact, elementwise bound)."""
    p = np.abs(va) @ np.abs(vb).T
    if old is not None:
        v, p = v + old, p + np.abs(old)
    if dtype == "bf16":
        return v, 2.0 ** -8 * np.abs(v) + 2.0 ** -9 * p
    return v, 2.0 ** -24 * np.abs(v) + (va.shape[1] / 32 + 64) * 2.0 ** -24 * p


def check_product(out, va, vb, dtype, old=None):
    v, tol = bound(va, vb, va @ vb.T, dtype, old)
    err = np.abs(out.double().cpu().numpy() - v)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    n = np.linalg.norm(v)
    return np.linalg.norm(err) / n if n else 0.0


SIZES = [(1, 1, 1), (1, 6144, 2048), (2, 17, 129), (16, 512, 2048), (17, 130, 1000), (33, 64, 128), (64, 300, 4096),
         (65, 15, 64), (128, 128, 128), (129, 257, 385), (300, 1, 700), (777, 1003, 501), (1024, 512, 256),
         (200, 300, 8192), (513, 2050, 640), (2100, 1100, 192), (2900, 2900, 100), (2817, 3000, 1301),
         (4096, 2048, 384), (1536, 5400, 2560)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_against_fp64(m, n, k, dtype):
    a, va = operand(m, k, 11)
    b, vb = operand(n, k, 12, "tiles")
    out = mh().fp8_matmul(a, b, out_dtype=DT[dtype])
    assert out.shape == (m, n) and out.dtype == DT[dtype]
    rel = check_product(out, va, vb, dtype)
    # over a whole product the errors are far below the elementwise bounds:
    # a rounding's relative error is at most 2^-8 (2^-24) each
    assert rel <= (2.0 ** -8 if dtype == "bf16" else 1e-5)
    again = mh().fp8_matmul(a, b, out_dtype=DT[dtype])
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [64, 128, 129, 300, 400, 520, 700, 1100, 2300])
@pytest.mark.parametrize("m,n", [(9, 150), (200, 190), (640, 730), (1500, 1420), (3100, 3300), (4090, 3900)])
def test_product_at_every_tile_size_and_loop_length(m, n, k, dtype):
    """Tiles of 16, 64, 128, 192 x 256 and 256; 1 to 18 blocks of k: shorter than,
    as long as and longer than every ring, ending in a ragged block or not."""
    a, va = operand(m, k, 21)
    b, vb = operand(n, k, 22)
    check_product(mh().fp8_matmul(a, b, out_dtype=DT[dtype]), va, vb, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ab", [("rows", "rows"), ("tiles", "rows"), ("tiles", "tiles"), ("rows", "tiles")])
@pytest.mark.parametrize("m,n,k", [(40, 300, 700), (300, 260, 700), (140, 200, 5000), (640, 730, 300), (1400, 1500, 300),
                                   (3200, 3100, 300), (3900, 4050, 300)])
def test_product_of_block_kinds_accumulates(m, n, k, ab, dtype):
    a, va = operand(m, k, 13, ab[0], spread=False)
    b, vb = operand(n, k, 14, ab[1], spread=False)
    old = torch.from_numpy(np.random.default_rng(15).standard_normal((m, n)).astype(np.float32) * 30).cuda().to(DT[dtype])
    out = old.clone()
    got = mh().fp8_matmul(a, b, out=out, accumulate=True)
    assert got is out
    check_product(out, va, vb, dtype, old.double().cpu().numpy())
    mh().fp8_matmul(a, b, out=out)  # and without: the old values do not matter
    check_product(out, va, vb, dtype)
    out.fill_(float("nan"))
    mh().fp8_matmul(a, b, out=out)
    check_product(out, va, vb, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", [(3, 200, 256), (150, 203, 256), (150, 203, 6000), (640, 733, 300), (1400, 1433, 300),
                                   (3100, 3099, 200), (4000, 3999, 200)])
@pytest.mark.parametrize("extra,first", [(53, 0), (8, 0), (0, 1), (61, 8)])
def test_product_into_strided_rows_writes_nothing_else(m, n, k, extra, first, dtype):
    ld = n + extra
    a, va = operand(m, k, 16, spread=False)
    b, vb = operand(n, k, 17, spread=False)
    buf = torch.full((m * ld + 64,), 7.0, dtype=DT[dtype], device="cuda")
    out = buf[first:first + (m - 1) * ld + n].as_strided((m, n), (ld, 1), first)
    for acc in (False, True):
        old = out.double().cpu().numpy() if acc else None
        mh().fp8_matmul(a, b, out=out, accumulate=acc)
        check_product(out, va, vb, dtype, old)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[first:first + (m - 1) * ld + n].as_strided((m, n), (ld, 1), first).fill_(False)
    assert (buf[mask] == 7.0).all()
    # the place of out does not change the values
    assert torch.equal(mh().fp8_matmul(a, b, out_dtype=DT[dtype]), mh().fp8_matmul(a, b, out=out))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_product_of_empty_operands(dtype):
    e = lambda r, c: mh().Fp8Matrix.empty(r, c)  # noqa: E731
    for m in (3, 200, 70000):
        old = torch.full((m, 5), 2.0, device="cuda", dtype=DT[dtype])
        assert (mh().fp8_matmul(e(m, 0), e(5, 0), out=old, accumulate=True) == 2.0).all()
        assert (mh().fp8_matmul(e(m, 0), e(5, 0), out=old) == 0.0).all()
    assert mh().fp8_matmul(e(0, 128), e(5, 128), out_dtype=DT[dtype]).shape == (0, 5)
    assert mh().fp8_matmul(e(5, 128), e(0, 128), out_dtype=DT[dtype]).shape == (5, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", [(5, 150, 300), (140, 150, 300), (140, 150, 5000), (640, 730, 300), (1500, 1400, 300),
                                   (3100, 3200, 300), (3900, 4050, 300)])
def test_nan_and_overflow_stay_in_their_rows(m, n, k, dtype):
    g = torch.Generator("cuda").manual_seed(4)
    x, w = torch.randn(m, k, device="cuda", generator=g), torch.randn(n, k, device="cuda", generator=g)
    x[2, 7] = float("nan")
    x[3, 290] = float("inf")
    w[9, 150] = -float("inf")
    w[11] *= 2.0 ** 120
    x[4] *= 2.0 ** 120
    a, b = mh().fp8_quantize(x)[0], mh().fp8_quantize(w)[0]
    out = mh().fp8_matmul(a, b, out_dtype=DT[dtype]).double().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        va, vb = fo.values(*host(a), (m, k)), fo.values(*host(b), (n, k))
        v, p = va @ vb.T, np.abs(va) @ np.abs(vb).T
    # [4, 11]: products of both signs near 2^240, so partial sums in fp32 are
    # +inf and -inf, whose sum is NaN: not finite is all that fp32 sums promise
    rest = np.ones((m, n), bool)
    rest[4, 11] = False
    assert not np.isfinite(out[4, 11])
    assert np.array_equal(np.isnan(out)[rest], np.isnan(v)[rest])
    # where all magnitudes together stay below 2^127, no partial sum overflows
    # (2^120 times 5000 normal products does not: such results may be infinite)
    with np.errstate(invalid="ignore"):
        assert np.isfinite(out[rest & (p < 2.0 ** 127)]).all()
    assert (rest & (p < 2.0 ** 127)).sum() > (m - 4) * (n - 2) // 2


def test_product_of_long_rows_and_far_offsets():
    # codes past 2^31 bytes: 140000 rows of 16384; only some results are checked
    rows, k = 140000, 16384
    x = torch.randn(64, k, device="cuda")
    q, _ = mh().fp8_quantize(x)
    big = mh().Fp8Matrix.empty(rows, k)
    big.codes.view(torch.uint8).zero_()
    big.scales.view(torch.uint8).fill_(127)
    big.codes.view(torch.uint8)[-64:] = q.codes.view(torch.uint8)
    big.scales.view(torch.uint8)[-64:] = q.scales.view(torch.uint8)
    w, vw = operand(130, k, 18, spread=False)
    vx = fo.values(*host(q), (64, k))
    for dtype in ("bf16", "fp32"):
        out = mh().fp8_matmul(big, w, out_dtype=DT[dtype])
        check_product(out[-64:], vx, vw, dtype)
        assert not out[:-64].any()
        out = mh().fp8_matmul(w, big, out_dtype=DT[dtype])
        check_product(out[:, -64:], vw, vx, dtype)
        one = mh().Fp8Matrix(w.codes[:3], w.scales[:3], (3, k))
        out = mh().fp8_matmul(one, big, out_dtype=DT[dtype])
        check_product(out[:, -64:], vw[:3], vx, dtype)


# ---- a plan's weights ---------------------------------------------------------------
SHAPES = [(300, 200), (128, 256), (300, 200), (1, 5), (513, 129)] + [(8 + i, 40 + 3 * i) for i in range(20)]


@pytest.mark.parametrize("transposed", [True, False])
def test_weights_of_a_plan(transposed):
    opt = mh().MuonH(SHAPES)  # more shape groups than one launch holds
    W = [values(r, c, 20 + i) for i, (r, c) in enumerate(SHAPES)]
    ws = opt.fp8_weights(transposed)
    ws.storage.fill_(0xA5)
    assert opt.quantize_weights(W, ws) is ws
    assert len(ws.transposed) == (len(SHAPES) if transposed else 0)
    for i, w in enumerate(W):
        x64 = w.double().cpu().numpy()
        check_matrix(ws.weights[i], x64, "tiles")
        if transposed:
            check_matrix(ws.transposed[i], x64.T, "tiles")


def test_step_leaves_its_weights_quantized():
    shapes = [(256, 384), (130, 70), (256, 384)]
    def state():
        W = [values(r, c, 30 + i) * 1e-3 for i, (r, c) in enumerate(shapes)]
        return W, [torch.randn(s, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) for i, s in
                   enumerate(shapes)], [torch.zeros(s, device="cuda") for s in shapes]
    for name in ("step", "step_muon_wd"):
        opt = mh().MuonH(shapes)
        W0, G, M0 = state()
        W1, _, M1 = state()
        opt.init(W0)
        ws = opt.fp8_weights()
        getattr(opt, name)(W0, G, M0, 0.02)
        getattr(opt, name)(W1, G, M1, 0.02, fp8=ws)
        for i in range(len(shapes)):
            assert torch.equal(W0[i], W1[i]) and torch.equal(M0[i], M1[i])
            check_matrix(ws.weights[i], W1[i].double().cpu().numpy(), "tiles")
            check_matrix(ws.transposed[i], W1[i].double().cpu().numpy().T, "tiles")


def test_binding_refusals_enqueue_nothing():
    m = mh()
    opt, other = m.MuonH([(64, 64)]), m.MuonH([(64, 65)])
    W = [torch.randn(64, 64, device="cuda")]
    M, G = [torch.zeros_like(W[0])], [torch.ones_like(W[0])]
    opt.init(W)
    W0 = W[0].clone()
    ws = opt.fp8_weights()
    with pytest.raises(TypeError):
        opt.step(W, G, M, 0.02, fp8=[W[0]])
    with pytest.raises(ValueError, match="shapes"):
        opt.step(W, G, M, 0.02, fp8=other.fp8_weights())
    inside = ws.storage[:64 * 64 * 4].view(torch.float32).view(64, 64) if ws.storage.numel() >= 64 * 64 * 4 else None
    if inside is not None:
        with pytest.raises(m.MuonHAliasError):
            opt.quantize_weights([inside], ws)
    assert torch.equal(W[0], W0)
    x = torch.randn(100, 200, device="cuda")
    q, _ = m.fp8_quantize(x)
    for bad in (x.t(), x[:, ::2], x.expand(3, 100, 200), x[0]):
        with pytest.raises(ValueError):
            m.fp8_quantize(bad)
    with pytest.raises(ValueError):
        m.fp8_quantize(x[:1].expand(100, 200))  # rows overlap
    with pytest.raises(ValueError):
        m.fp8_quantize(x, block="columns")
    with pytest.raises(ValueError):
        m.fp8_quantize(x, forms="all")
    with pytest.raises(ValueError, match="out_t"):
        m.fp8_quantize(x, out_t=m.Fp8Matrix.empty(200, 100))
    with pytest.raises(ValueError, match="out must"):
        m.fp8_quantize(x, out=m.Fp8Matrix.empty(100, 201))
    with pytest.raises(ValueError, match="columns"):
        m.fp8_matmul(q, m.Fp8Matrix.empty(5, 201))
    with pytest.raises(ValueError, match="needs out"):
        m.fp8_matmul(q, q, accumulate=True)
    with pytest.raises(TypeError):
        m.fp8_matmul(q, q, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        m.fp8_matmul(q, q, out=torch.empty(100, 100, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError, match="out must"):
        m.fp8_matmul(q, q, out=torch.empty(100, 101, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        m.fp8_matmul(q, q, out=torch.empty(100, 100, device="cuda").t())
    with pytest.raises(m.MuonHError):  # out inside an operand's codes
        m.fp8_matmul(q, q, out=q.codes.view(torch.uint8).reshape(-1)[:100 * 100 * 2].view(torch.bfloat16).view(100, 100))


# ---- together ------------------------------------------------------------------------
def test_linear_layers_gradients():
    """Y = X W^T, dX = dY W, dW = dY^T X on quantized values, against the
    formula's and against differences of f(X, W) = <dY, X W^T> in fp64."""
    m = mh()
    t, n, k = 300, 260, 200
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(t, k, device="cuda", generator=g).to(torch.bfloat16)
    dy = (torch.randn(t, n, device="cuda", generator=g) * 1e-3).to(torch.bfloat16)
    opt = m.MuonH([(n, k)])
    W = [torch.randn(n, k, device="cuda", generator=g) * 0.05]
    ws = opt.quantize_weights(W, opt.fp8_weights())
    qx, qxt = m.fp8_quantize(x, forms="both")
    qd, qdt = m.fp8_quantize(dy, forms="both")
    y = m.fp8_matmul(qx, ws.weights[0], out_dtype=torch.float32)
    dx = m.fp8_matmul(qd, ws.transposed[0], out_dtype=torch.float32)
    dw = m.fp8_matmul(qdt, qxt, out_dtype=torch.float32)
    val = lambda q: fo.values(*host(q), q.shape, q.block)  # noqa: E731
    vx, vd, vw = val(qx), val(qd), val(ws.weights[0])
    assert np.array_equal(val(ws.transposed[0]), vw.T)  # one set of values, both orientations
    vdt, vxt = val(qdt), val(qxt)
    check_product(y, vx, vw, "fp32")
    check_product(dx, vd, vw.T, "fp32")
    check_product(dw, vdt, vxt, "fp32")
    rng = np.random.default_rng(9)
    # f is linear in each argument, so central differences are exact up to
    # fp64 rounding, and a directional derivative <grad, d> adds up the
    # elementwise bounds
    for grad, f, at, bounds in (
            (dx, lambda z: np.sum(vd * (z @ vw.T)), vx, bound(vd, vw.T, vd @ vw, "fp32")[1]),
            (dw, lambda z: np.sum(vdt.T * (vxt.T @ z.T)), vw, bound(vdt, vxt, vdt @ vxt.T, "fp32")[1])):
        d = rng.standard_normal(at.shape)
        diff = (f(at + 0.5 * d) - f(at - 0.5 * d))
        got = np.sum(grad.double().cpu().numpy() * d)
        assert abs(got - diff) <= np.sum(bounds * np.abs(d)) + 1e-9 * abs(diff)


def train(m, opt, ws, W, M, G, x, dy, steps, bufs):
    """Two micro-batches of one layer's products, then the step; all buffers given."""
    qx, qxt, qd, qdt, y, dx = bufs
    for _ in range(steps):
        for half in range(2):
            m.fp8_quantize(x[half], forms="both", out=qx, out_t=qxt)
            m.fp8_quantize(dy[half], forms="both", out=qd, out_t=qdt)
            m.fp8_matmul(qx, ws.weights[0], out=y)
            m.fp8_matmul(qd, ws.transposed[0], out=dx)
            m.fp8_matmul(qdt, qxt, out=G[0], accumulate=half > 0)
        opt.step(W, G, M, 0.02, fp8=ws)


@pytest.mark.parametrize("t,n,k", [(256, 384, 256), (1000, 130, 200)])
def test_training_steps_replay_in_a_graph_and_on_streams(t, n, k):
    """Quantize, the three products, the step with 8-bit weights: captured and
    replayed (eager work between the replays), and run eagerly on a stream
    of its own beside another one, all bit for bit the same."""
    m = mh()
    g = torch.Generator("cuda").manual_seed(6)
    x = [torch.randn(t, k, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    dy = [torch.randn(t, n, device="cuda", generator=g) * 1e-2 for _ in range(2)]
    W0 = torch.randn(n, k, device="cuda", generator=g) * 0.05

    def make():
        opt = m.MuonH([(n, k)])
        W, M, G = [W0.clone()], [torch.zeros(n, k, device="cuda")], [torch.zeros(n, k, device="cuda")]
        opt.init(W)
        ws = opt.quantize_weights(W, opt.fp8_weights())
        bufs = (m.Fp8Matrix.empty(t, k), m.Fp8Matrix.empty(k, t), m.Fp8Matrix.empty(t, n), m.Fp8Matrix.empty(n, t),
                torch.empty(t, n, device="cuda", dtype=torch.bfloat16), torch.empty(t, k, device="cuda"))
        return opt, ws, W, M, G, bufs

    def snap(W, M, G, ws, bufs):
        # the matrices of the set, not its storage: that has gaps between them
        held = [v.view(torch.uint8) for q in ws.weights + ws.transposed for v in (q.codes, q.scales)]
        return [v.clone() for v in (W[0], M[0], G[0], bufs[4], bufs[5], *held)]

    opt, ws, W, M, G, bufs = make()
    want = []
    for _ in range(4):
        train(m, opt, ws, W, M, G, x, dy, 1, bufs)
        torch.cuda.synchronize()
        want.append(snap(W, M, G, ws, bufs))

    opt, ws, W, M, G, bufs = make()
    train(m, opt, ws, W, M, G, x, dy, 1, bufs)  # builds the pointer arrays
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train(m, opt, ws, W, M, G, x, dy, 1, bufs)
    torch.cuda.synchronize()
    for r in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(snap(W, M, G, ws, bufs), want[r])), f"replay {r}"
        float(torch.randn(1 << 20, device="cuda").sum())  # eager work between the replays
        m.fp8_matmul(bufs[3], bufs[1], out_dtype=torch.float32)
        torch.cuda.synchronize()

    pair = [(torch.cuda.Stream(), make()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (opt, ws, W, M, G, bufs) in pair:
            with torch.cuda.stream(s):
                train(m, opt, ws, W, M, G, x, dy, 1, bufs)
    torch.cuda.synchronize()
    for s, (opt, ws, W, M, G, bufs) in pair:
        assert all(torch.equal(u, v) for u, v in zip(snap(W, M, G, ws, bufs), want[3]))
