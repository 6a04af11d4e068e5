"""RMS norm on the GPU against the fp64 oracle, element by element.

u = 2^-24, half a step of fp32. Bounds, from the operations:
  h: bit for bit the fp32 sum rounded to its type.
  r: a sum of squares in fp32, in which a term meets at most D roundings (its own
     square, 8 in its vector, up to 4 vectors, 6 among the lanes of a wave, 16
     waves; rows over 32768 columns also cols/8192 turns): D u of the sum, half of it in r, then
     inverse count, product, eps (3 u, half) and the inverse root (1 ulp = 2 u).
  y: two more roundings, then its type's.
  dh = r (g - n mean) + dres: mean as r's sum with two more roundings, D + 6;
     per entry 5 roundings on either term, 2 on the sum, 1 with dres, then its type's.
  dw: a sum over rows of products of 2 roundings, in which a term meets the
     rows that its lane takes, those of its workgroup, and the partial sums.
8 bits: a code lies between the codes of y (1 +- bound), a scale between the
  scales of the maximum (1 +- bound).
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import fp8_oracle as fo
from oracle import norm_oracle as no

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def mh():
    import orthogonalized_updates_amd
    return orthogonalized_updates_amd


def f64(t):
    return t.double().cpu().numpy()


def depth(cols):
    return 1 + 8 + 4 + 6 + 16 + cols / 8192


def tol_r(cols):
    return (0.5 * depth(cols) + 1.5 + 2) * U


def values(rows, cols, seed, dtype="fp32", scale=1.0):
    rng = np.random.default_rng((seed, rows, cols))
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-8, 8, (rows, 1))) * np.exp2(rng.integers(-3, 4, (1, cols)))
    return torch.from_numpy((x * scale).astype(np.float32)).to(DT[dtype]).cuda()


def weights(cols, seed=0):
    return torch.from_numpy((1 + 0.3 * np.random.default_rng((seed, cols)).standard_normal(cols)).astype(np.float32)).cuda()


def check_y(y, r, h, w, eps=EPS):
    want, wr = no.forward(f64(h), f64(w), eps)
    t = tol_r(h.shape[1])
    assert (np.abs(f64(r) - wr) <= t * wr).all()
    err = np.abs(f64(y) - want)
    assert (err <= (t + 2 * U + HALF[y.dtype]) * np.abs(want) + 1e-44).all(), err.max()


def check_codes(q, y64, rel):
    """q holds y64, each entry and each maximum known to `rel`."""
    rows, cols = q.shape
    codes, scales = q.codes.view(torch.uint8).cpu().numpy(), q.scales.view(torch.uint8).cpu().numpy()
    nb = -(-cols // 128)
    assert not codes[:, cols:].any() and not scales[:, nb:].any()
    lo, hi = fo.quantize(y64 * (1 - rel))[1], fo.quantize(y64 * (1 + rel))[1]
    assert ((scales == lo) | (scales == hi)).all()
    s = np.ldexp(1.0, scales[:, :nb].astype(np.int64) - 127).repeat(128, 1)[:, :cols]
    got = fo.decode(codes[:, :cols])
    # both ends rounded to e4m3; the larger one may round past 448 only where the scale does not fit it
    a, b = fo.decode(fo.encode(np.clip(y64 * (1 - rel) / s, -448, 448))), fo.decode(fo.encode(np.clip(y64 * (1 + rel) / s, -448, 448)))
    assert ((np.minimum(a, b) <= got) & (got <= np.maximum(a, b))).all()


def add(x, res):
    return x if res is None else (x.float() + res.float()).to(res.dtype)


SIZES = [(1, 1), (1, 2048), (3, 7), (2, 128), (17, 129), (300, 128), (5, 512), (257, 520), (64, 1000), (300, 1001), (300, 1536),
         (129, 2048), (258, 2048), (7, 2056), (300, 4096), (33, 8192), (3, 8200), (40, 16384), (5, 20000), (2, 32768), (3, 40001)]


@pytest.mark.parametrize("types", [("bf16", None), ("fp32", None), ("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm(rows, cols, types):
    x, w = values(rows, cols, 1, types[0]), weights(cols)
    res = None if types[1] is None else values(rows, cols, 2, types[1])
    ref = add(x, res)
    for out_dtype in (None, torch.float32, torch.bfloat16):
        y, h, r = mh().rms_norm(x, w, residual=res, eps=EPS, out_dtype=out_dtype)
        assert y.dtype == (out_dtype or ref.dtype) and h.dtype == ref.dtype and r.dtype == torch.float32
        assert torch.equal(h, ref) and (res is not None or h is x)
        check_y(y, r, ref, w)


@pytest.mark.parametrize("types", [("bf16", None), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_in_8_bits(rows, cols, types):
    x, w = values(rows, cols, 3, types[0]), weights(cols, 1)
    res = None if types[1] is None else values(rows, cols, 4, types[1])
    ref = add(x, res)
    want, wr = no.forward(f64(ref), f64(w), EPS)
    rel = tol_r(cols) + 2 * U
    first = None
    for forms in ("plain", "transposed", "both"):
        q, qt, h, r = mh().rms_norm_fp8(x, w, residual=res, eps=EPS, forms=forms)
        assert (q is None) == (forms == "transposed") and (qt is None) == (forms == "plain")
        assert torch.equal(h, ref) and (np.abs(f64(r) - wr) <= tol_r(cols) * wr).all()
        if q is not None:
            check_codes(q, want, rel)
        if qt is not None:
            check_codes(qt, want.T, rel)
        # one r for all forms, so the same codes whichever are asked for
        if forms == "plain":
            first = q
        elif q is not None:
            assert torch.equal(q.codes.view(torch.uint8), first.codes.view(torch.uint8))
            assert torch.equal(q.scales.view(torch.uint8), first.scales.view(torch.uint8))


# 64 lanes with a vector each: more than 256 rows of 129 to 512 columns
LANES_64 = [(300, 129), (300, 500), (257, 512), (261, 385)]


@pytest.mark.parametrize("types", [("bf16", None), ("fp32", None), ("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols", LANES_64)
def test_norm_by_64_lanes(rows, cols, types):
    test_norm(rows, cols, types)
    test_norm_in_8_bits(rows, cols, types)


# more rows than a launch's workgroups take at once, by less than ENDS
ENDS = 12
TALL = [((4 << 20) + 9, 130), ((4 << 20) + 9, 515), ((4 << 20) + 9, 1025), ((1 << 20) + 5, 1537), ((1 << 20) + 5, 2049), ((1 << 20) + 5, 4097),
        ((1 << 20) + 5, 8193), ((1 << 20) + 5, 16385), ((1 << 20) + 5, 32769)]


def tall(rows, cols, seed, rest, scale=1.0):
    """A bf16 matrix with values in its first and last ENDS rows, and these."""
    if torch.cuda.mem_get_info()[0] < 4 * rows * cols + rest:
        torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 4 * rows * cols + rest:
        pytest.skip("not enough free memory")
    x, ends = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"), values(2 * ENDS, cols, seed, "bf16", scale)
    x[:ENDS], x[-ENDS:] = ends[:ENDS], ends[ENDS:]
    return x, ends


def both_ends(t):
    return torch.cat([t[:ENDS], t[-ENDS:]])


@pytest.mark.parametrize("rows,cols", TALL)
def test_rows_past_the_most_workgroups(rows, cols):
    x, ends = tall(rows, cols, 1, 8 << 30)
    w = weights(cols).abs()  # so that zeros have no sign
    want = no.forward(f64(ends), f64(w), EPS)[0]
    q, _, _, r = mh().rms_norm_fp8(x, w, eps=EPS)
    assert float((r[ENDS:-ENDS] - 1e3).abs().max()) <= tol_r(cols) * 1e3
    codes, scales = (both_ends(t.view(torch.uint8)) for t in (q.codes, q.scales))
    check_codes(mh().Fp8Matrix(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), (2 * ENDS, cols)), want, tol_r(cols) + 2 * U)
    rest = q.codes.view(torch.uint8)[ENDS:-ENDS]
    assert int(rest.amax()) == 0
    del q, rest
    y, _, r = mh().rms_norm(x, w, eps=EPS)
    check_y(both_ends(y), both_ends(r), ends, w)
    assert float(y[ENDS:-ENDS].amax()) == float(y[ENDS:-ENDS].amin()) == 0


# more rows than the gradient's workgroups take at once: dw is summed over a workgroup's sets of rows
TURNS = [(33000, 128), (32800, 77), (2100, 300), (2100, 1001), (2100, 1500), (2100, 2047), (1030, 4095), (1030, 8190), (520, 16384), (515, 12001),
         (70, 20000), (67, 16391)]


@pytest.mark.parametrize("types", [("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols", TURNS)
def test_gradient_over_further_rows(rows, cols, types):
    test_gradient(rows, cols, types)


def test_gradient_of_long_rows_past_the_most_workgroups():
    rows, cols = (1 << 20) + 5, 16387
    (h, hends), (dy, dends) = tall(rows, cols, 1, 48 << 30), tall(rows, cols, 2, 8 << 30, 1e-3)
    w, r = weights(cols), torch.full((rows,), 1e3, device="cuda")
    rends = torch.from_numpy(no.forward(f64(hends), f64(w), EPS)[1].astype(np.float32)).cuda()
    r[:ENDS], r[-ENDS:] = rends[:ENDS], rends[ENDS:]
    dh, dw = mh().rms_norm_backward(dy, h, w, r, out=dy)
    check_back(both_ends(dh), dw, dends, hends, w, rends, None)
    assert float(dh[ENDS:-ENDS].amax()) == float(dh[ENDS:-ENDS].amin()) == 0


def check_back(dh, dw, dy, h, w, r, res):
    rows, cols = h.shape
    d64, h64, w64, r64 = f64(dy), f64(h), f64(w), f64(r)[:, None]
    want, wdw = no.backward(d64, h64, w64, f64(r), None if res is None else f64(res))
    g, n = np.abs(d64 * w64), np.abs(h64 * r64)
    m = np.mean(g * n, axis=1, keepdims=True)
    tol = U * (7 * r64 * g + (depth(cols) + 6 + 7) * r64 * n * m) + HALF[dh.dtype] * np.abs(want)
    if res is not None:
        tol += U * np.abs(f64(res)) + U * np.abs(want)
    err = np.abs(f64(dh) - want)
    assert (err <= tol + 1e-44).all(), (err / (tol + 1e-44)).max()
    per = 16 if cols <= 128 else 4 if cols <= 2048 else 1
    blocks = min(rows, 64) if cols > 16384 else min(-(-rows // per), 2048 if cols <= 128 else 1024 if 2048 < cols <= 8192 else 512)
    terms = 3 + math.ceil(rows / (blocks * (per if cols <= 16384 else 1))) + 16 + blocks / 32 + 32
    assert (np.abs(f64(dw) - wdw) <= U * terms * np.sum(np.abs(d64) * n, axis=0) + 1e-44).all()


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols", SIZES + [(5000, 64), (9000, 128), (2500, 1024)])
def test_gradient(rows, cols, types):
    dy, h, w = values(rows, cols, 5, types[0], 1e-3), values(rows, cols, 6, types[1]), weights(cols, 2)
    r = torch.from_numpy(no.forward(f64(h), f64(w), EPS)[1].astype(np.float32)).cuda()
    for res in (None, values(rows, cols, 7, types[1], 1e-3)):
        dh, dw = mh().rms_norm_backward(dy, h, w, r, dresidual=res)
        assert dh.dtype == h.dtype and dw.dtype == torch.float32
        check_back(dh, dw, dy, h, w, r, res)
        again = mh().rms_norm_backward(dy, h, w, r, dresidual=res)
        assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
    old = weights(cols, 9)
    got = mh().rms_norm_backward(dy, h, w, r, dresidual=res, dweight=old.clone(), accumulate=True)[1]
    assert torch.equal(got, old + dw)


def test_gradient_against_differences():
    """Of the kernel's own fp32 results: a difference of sums S over 2^-6 steps holds
    about 2^-24 * sum|t y| / 2^-6 of rounding and step^2 / 6 of curvature: 1e-3 covers both here."""
    rows, cols, step = 3, 40, 2.0 ** -6
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).cuda()
    t = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).cuda()
    w = weights(cols, 3)
    dh, dw = mh().rms_norm_backward(t, x, w, mh().rms_norm(x, w, eps=0.1)[2])

    def f(x, w):
        return float((t.double() * mh().rms_norm(x, w, eps=0.1)[0].double()).sum())

    for i in range(rows):
        for j in range(0, cols, 7):
            d = torch.zeros_like(x)
            d[i, j] = step
            assert abs((f(x + d, w) - f(x - d, w)) / (2 * step) - float(dh[i, j])) < 1e-3
    for j in range(0, cols, 7):
        d = torch.zeros_like(w)
        d[j] = step
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * step) - float(dw[j])) < 1e-3


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("cols,ld,first", [(300, 301, 1), (2048, 2050, 3), (128, 640, 0), (5000, 5003, 1), (2048, 4096, 2048)])
def test_strides_and_untouched_neighbours(cols, ld, first, dtype):
    """Rows inside wider ones, at odd offsets; what lies between them stays."""
    rows = 21

    def inside(seed, fill=None):
        base = values(rows + 1, ld, seed, dtype).reshape(-1)
        if fill is not None:
            base.fill_(fill)
        return base, base.as_strided((rows, cols), (ld, 1), first)

    (_, x), (_, res), w = inside(1), inside(2), weights(cols, 4)
    (by, y), (bh, h) = inside(3, 7.0), inside(3, 7.0)
    got = mh().rms_norm(x, w, residual=res, eps=EPS, out=y, residual_out=h)
    assert got[0] is y and got[1] is h
    assert torch.equal(h, add(x, res))
    check_y(y, got[2], h.clone(), w)
    q, qt, _, _ = mh().rms_norm_fp8(x, w, residual=res, eps=EPS, forms="both", residual_out=h)
    want = no.forward(f64(h), f64(w), EPS)[0]
    check_codes(q, want, tol_r(cols) + 2 * U)
    check_codes(qt, want.T, tol_r(cols) + 2 * U)
    (_, dy), (_, dres), (bd, dh) = inside(4), inside(5), inside(3, 7.0)
    _, dw = mh().rms_norm_backward(dy, h, w, got[2], dresidual=dres, out=dh)
    check_back(dh.clone(), dw, dy, h, w, got[2], dres)
    for base in (by, bh, bd):
        keep = torch.ones_like(base, dtype=torch.bool)
        keep.as_strided((rows, cols), (ld, 1), first).fill_(False)
        assert (base[keep] == 7.0).all()


def test_columns_of_one_wide_buffer():
    """Inputs and outputs side by side in the same rows."""
    rows, cols = 70, 256
    buf = values(rows, 5 * cols, 1, "bf16")
    x, res, h, y, dh = (buf[:, i * cols:(i + 1) * cols] for i in range(5))
    w = weights(cols)
    want = mh().rms_norm(x.contiguous(), w, residual=res.contiguous())
    got = mh().rms_norm(x, w, residual=res, residual_out=h, out=y)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    back = mh().rms_norm_backward(y, h, w, got[2], dresidual=res, out=dh)
    again = mh().rms_norm_backward(want[0], want[1], w, want[2], dresidual=res.contiguous())
    assert torch.equal(dh, again[0]) and torch.equal(back[1], again[1])
    with pytest.raises(mh().MuonHError) as e:
        mh().rms_norm(x, w, residual=res, residual_out=buf[:, cols - 1:2 * cols - 1])
    assert e.value.status == mh().MUONH_EALIAS


@pytest.mark.parametrize("rows,cols", [(5, 2048), (300, 128), (400, 1001), (3, 40000)])
def test_in_place(rows, cols):
    x, res, w = values(rows, cols, 1, "bf16"), values(rows, cols, 2, "bf16"), weights(cols)
    y, h, r = mh().rms_norm(x, w, residual=res)
    for target in ("res", "x"):
        a, b = x.clone(), res.clone()
        got = mh().rms_norm(a, w, residual=b, residual_out=b if target == "res" else a)
        assert all(torch.equal(p, q) for p, q in zip(got, (y, h, r)))
    q, qt, _, _ = mh().rms_norm_fp8(x, w, residual=res, forms="both")
    b = res.clone()
    p, pt, _, _ = mh().rms_norm_fp8(x, w, residual=b, forms="both", residual_out=b, out=mh().Fp8Matrix.empty(rows, cols),
                                    out_t=mh().Fp8Matrix.empty(cols, rows))
    for m, n in ((p, q), (pt, qt)):
        assert torch.equal(m.codes.view(torch.uint8), n.codes.view(torch.uint8))
    dy, dres = values(rows, cols, 3, "bf16"), values(rows, cols, 4, "bf16")
    want = mh().rms_norm_backward(dy, h, w, r, dresidual=dres)
    a, b = dy.clone(), dres.clone()
    assert torch.equal(mh().rms_norm_backward(a, h, w, r, dresidual=dres, out=a)[0], want[0])
    assert torch.equal(mh().rms_norm_backward(dy, h, w, r, dresidual=b, out=b)[0], want[0])


@pytest.mark.parametrize("rows,cols", [(20, 128), (20, 2048), (300, 2048), (4, 5000), (3, 40000)])
def test_zeros_infinities_and_nan_stay_in_their_rows(rows, cols):
    x, w = values(rows, cols, 1), weights(cols)
    x[0] = 0
    x[1, cols // 2] = float("nan")
    x[2, cols - 1] = float("inf")
    x[3 % rows, :] = 1e30 if rows > 3 else x[3 % rows, :]
    y, _, r = mh().rms_norm(x, w, eps=EPS)
    assert (y[0] == 0).all() and abs(float(r[0]) - 1e3) <= tol_r(cols) * 1e3
    assert y[1].isnan().all() and r[1].isnan()
    assert float(r[2]) == 0 and y[2, -1].isnan() and (y[2, :-1] == 0).all()
    if rows > 3:
        assert float(r[3]) == 0 and (y[3] == 0).all()  # its mean square is past fp32's range
    if rows > 4:
        check_y(y[4:], r[4:], x[4:], w)
    q, qt, _, _ = mh().rms_norm_fp8(x, w, eps=EPS, forms="both")
    codes = q.codes.view(torch.uint8)[:, :cols]
    assert (codes[0] & 127 == 0).all() and ((codes[1] & 127) == 127).all()
    assert (codes[2, :-1] & 127 == 0).all() and int(codes[2, -1]) & 127 == 127
    assert not q.codes.view(torch.uint8)[:, cols:].any()
    # a NaN of one row in a column's block does not count for its scale, nor spread
    ct = qt.codes.view(torch.uint8)[:, :rows].t()
    assert ((ct[1] & 127) == 127).all() and not qt.codes.view(torch.uint8)[:, rows:].any()
    if rows > 4:
        assert not ((ct[4:] & 127) == 127).any()
    y0, _, r0 = mh().rms_norm(x[:1], w, eps=0.0)
    assert float(r0[0]) == math.inf and y0.isnan().all()  # 0 / 0
    dy = values(rows, cols, 2)
    dh, dw = mh().rms_norm_backward(dy, x, w, r)
    assert dh[1].isnan().all() and not dh[0].isnan().any() and dw.isnan().all()
    if rows > 4:
        assert not dh[4:].isnan().any()


def test_padding_of_8_bit_rows_is_zero_whatever_the_factors():
    """A last row whose r is infinite, a last column whose weight is: neither reaches the padding."""
    x, w = values(130, 200, 1), weights(200)
    x[-1] = 0
    w[-1] = float("inf")
    q, qt, _, _ = mh().rms_norm_fp8(x, w, eps=0.0, forms="both")
    for m in (q, qt):
        assert not m.codes.view(torch.uint8)[:, m.shape[1]:].any()
    p = mh().rms_norm_fp8(x, w, eps=0.0)[0]
    assert not p.codes.view(torch.uint8)[:, 200:].any()


def test_no_rows():
    x, w = torch.empty(0, 300, device="cuda"), weights(300)
    y, h, r = mh().rms_norm(x, w)
    assert y.shape == (0, 300) and r.shape == (0,)
    assert mh().rms_norm_fp8(x, w, forms="both")[1].shape == (300, 0)
    old = weights(300, 5)
    assert (mh().rms_norm_backward(x, x, w, r)[1] == 0).all()
    assert torch.equal(mh().rms_norm_backward(x, x, w, r, dweight=old.clone(), accumulate=True)[1], old)


def test_offsets_past_32_bits():
    ld = (1 << 30) + 8
    x = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    v = x.as_strided((3, 64), (ld, 1))
    v.copy_(values(3, 64, 1, "bf16"))
    w = weights(64)
    y, h, r = mh().rms_norm(v, w, eps=EPS)
    check_y(y, r, v.contiguous(), w)
    dy, h = values(3, 64, 2, "bf16"), v.contiguous()
    dh, dw = mh().rms_norm_backward(dy, h, w, r, dresidual=v, out=v)
    check_back(dh.contiguous(), dw, dy, h, w, r, h)


def test_python_refuses():
    m, x, w = mh(), values(4, 8, 1), weights(8)
    r = torch.ones(4, device="cuda")
    for call in (lambda: m.rms_norm(x, w[:7]), lambda: m.rms_norm(x, w.cpu()), lambda: m.rms_norm(x[0], w),
                 lambda: m.rms_norm(x.t(), weights(4)), lambda: m.rms_norm(x, w, residual=x[:3]),
                 lambda: m.rms_norm(x, w, residual_out=x), lambda: m.rms_norm(x, w, out=x[:, :7]),
                 lambda: m.rms_norm(x[:1].expand(4, 8), w), lambda: m.rms_norm_fp8(x, w, out=m.Fp8Matrix.empty(8, 4)),
                 lambda: m.rms_norm_backward(x, x, w, r[:3]), lambda: m.rms_norm_backward(x, x, w, r, accumulate=True)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: m.rms_norm(x, w.double()), lambda: m.rms_norm(x.half(), w), lambda: m.rms_norm(x, w, out_dtype=torch.half),
                 lambda: m.rms_norm(x, w, residual=x, residual_out=x.bfloat16()), lambda: m.rms_norm(x, w, out=x.bfloat16(), out_dtype=torch.float32),
                 lambda: m.rms_norm_backward(x, x, w, r, dresidual=x.bfloat16()), lambda: m.rms_norm_backward(x, x, w, r, out=x.bfloat16())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: m.rms_norm(x, w, out=x), lambda: m.rms_norm_backward(x.clone(), x, w, r, out=x)):
        with pytest.raises(m.MuonHError) as e:
            call()
        assert e.value.status == m.MUONH_EALIAS


def test_captured_graph_and_other_stream():
    x, res, w = values(700, 2048, 1, "bf16"), values(700, 2048, 2, "bf16"), weights(2048)
    dy, dres = values(700, 2048, 3, "bf16", 1e-3), values(700, 2048, 4, "bf16", 1e-3)

    def run():
        q, qt, h, r = mh().rms_norm_fp8(x, w, residual=res, forms="both")
        y = mh().rms_norm(h, w)[0]
        dh, dw = mh().rms_norm_backward(dy, h, w, r, dresidual=dres)
        return [q.codes.view(torch.uint8), qt.codes.view(torch.uint8), q.scales.view(torch.uint8), qt.scales.view(torch.uint8),
                h, r, y, dh, dw]

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = run()
    side = torch.cuda.Stream()
    for i in range(3):
        x.copy_(values(700, 2048, 10 + i, "bf16"))
        dy.copy_(values(700, 2048, 20 + i, "bf16", 1e-3))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = run()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(other, want))
