"""Microscaled 4-bit operators on the GPU against the fp64 oracle.

Quantization is defined bit for bit: codes, scales and padding must be equal, and
dequantized values too.

Products: where scales do not change along k, every product is a whole number of
quarters times one power of two, and sums stay below 2^24 of them: results are exact
in fp32 in any order. Otherwise, element by element, with v the exact value and
P = sum_k |a_k b_k|: the sums of groups of 32 are exact, and an instruction of 4 groups
adds at most 4 times, each off by at most a step (2^-23, whatever the direction of its rounding); up
to 16 partial sums, 8 waves' sums and the old value follow: (8 ceil(k/128) + 64) 2^-24 P, and half a
step of the result's type on |v|.
"""
from __future__ import annotations

import copy

import numpy as np
import pytest

from oracle import fp4_oracle as fo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {"fp32": U, "bf16": 2.0 ** -8}


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def mh():
    import orthogonalized_updates_amd
    return orthogonalized_updates_amd


def values(rows, cols, seed, dtype="fp32"):
    rng = np.random.default_rng((seed, rows, cols))
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1))) * np.exp2(rng.integers(-6, 7, (1, cols)))
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()


def special(rows, cols, seed, dtype):
    """NaN, infinities, zero groups, halfway values, full-scale and tiny ones."""
    x = values(rows, cols, seed, dtype)
    rng = np.random.default_rng(seed)
    g = fo.GRID
    pool = np.concatenate([g, (g[1:] + g[:-1]) / 2, -g, -(g[1:] + g[:-1]) / 2, [6 * 2.0 ** 7, 6.5 * 2.0 ** -20, 2.0 ** -126, 2.0 ** -133, 3.3e38, -0.0, 0.0]])
    x = torch.where(torch.from_numpy(rng.random((rows, cols)) < 0.4).cuda(),
                    torch.from_numpy(rng.choice(pool, (rows, cols)).astype(np.float32)).to(x.dtype).cuda(), x)
    bad = rng.random((rows, cols)) < 0.004
    x = torch.where(torch.from_numpy(bad).cuda(), torch.from_numpy(rng.choice([np.nan, np.inf, -np.inf], (rows, cols)).astype(np.float32)).to(x.dtype).cuda(), x)
    x[::3, :64] = 0.0
    return x


def host(m):
    return m.codes.view(torch.uint8).cpu().numpy(), m.scales.view(torch.uint8).cpu().numpy()


def check_matrix(m, x64):
    codes, scales = host(m)
    want_c, want_s = fo.quantize(x64)
    assert np.array_equal(scales, want_s)
    got, want = fo.unpack(codes), want_c
    # a zero's sign is the source's, which fp64 keeps; groups that are not finite hold zero codes
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (600, 1), (3, 640), (31, 33), (127, 129), (128, 128), (129, 300), (257, 513), (300, 1001), (640, 520)])
def test_quantize_is_the_definition(rows, cols, dtype):
    for x in (values(rows, cols, 5, dtype), special(rows, cols, 6, dtype)):
        q, qt = mh().fp4_quantize(x, forms="both")
        x64 = x.double().cpu().numpy()
        check_matrix(q, x64)
        check_matrix(qt, x64.T)
        for forms in ("plain", "transposed"):
            one = mh().fp4_quantize(x, forms=forms)
            assert [o is None for o in one] == [forms == "transposed", forms == "plain"]
            for o, ref in zip(one, (q, qt)):
                if o is not None:
                    assert all(np.array_equal(a, b) for a, b in zip(host(o), host(ref)))
        for m, v in ((q, x64), (qt, x64.T)):
            want = fo.values(*host(m), m.shape)
            for t in (torch.float32, torch.bfloat16):
                got = m.dequantize(t)
                assert got.dtype == t and got.shape == m.shape
                want_t = torch.from_numpy(want.astype(np.float32)).cuda().to(t)  # exact, but past fp32's range infinite
                assert torch.equal(torch.nan_to_num(got.float(), nan=7e30), torch.nan_to_num(want_t.float(), nan=7e30))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_groups_around_every_border(dtype):
    """Maxima at, just below and just above 6 * 2^e for every e, and at the ends."""
    e = np.arange(-130, 127)
    top = np.ldexp(6.0, e)
    top = np.concatenate([top[top < 3e38], [1e-45, 2.0 ** -149 * 3, 3.3895314e38]]).astype(np.float32)
    step = np.float32(2 ** -23 if dtype == "fp32" else 2 ** -7)
    a = np.concatenate([top, top * (1 - step / 2), np.minimum(top.astype(np.float64) * (1 + step), 3.38e38).astype(np.float32)])
    x = np.random.default_rng(2).uniform(-1, 1, (len(a), 96)).astype(np.float64) * a[:, None]
    x[:, 40] = a
    x = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    q, qt = mh().fp4_quantize(x, forms="both")
    check_matrix(q, x.double().cpu().numpy())
    check_matrix(qt, x.double().cpu().numpy().T)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_one_bad_entry_marks_its_group_only(dtype):
    kinds = [0x7f800001, 0x7fbfffff, 0x7fc00000, 0x7fffffff, 0x7f800000, 0xff800000, 0xffc00001, 0xff800001]
    if dtype == "bf16":
        kinds = [k >> 16 | (1 if k & 0xffff else 0) for k in kinds]
    base = values(len(kinds) * 40, 100, 3, dtype)
    bits = base.view(torch.int32 if dtype == "fp32" else torch.int16).cpu().numpy().copy()
    for i, k in enumerate(kinds):
        bits[40 * i + 5, 33 + i] = np.array(k, np.uint32).astype(np.int32) if dtype == "fp32" else np.array(k, np.uint16).astype(np.int16)
    x = torch.from_numpy(bits).cuda().view(DT[dtype])
    x64 = x.double().cpu().numpy()
    assert (~np.isfinite(x64)).sum() == len(kinds)
    q, qt = mh().fp4_quantize(x, forms="both")
    check_matrix(q, x64)
    check_matrix(qt, x64.T)
    assert int(q.dequantize().isnan().sum()) == 32 * len(kinds)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("ld,first", [(512, 0), (520, 8), (303, 0), (301, 1), (1024, 3)])
def test_quantize_of_strided_rows(ld, first, dtype):
    base = values(200, ld + 8, 7, dtype)
    x = base.reshape(-1)[first:first + 199 * ld + 300].as_strided((199, 300), (ld, 1))
    q, qt = mh().fp4_quantize(x, forms="both")
    check_matrix(q, x.double().cpu().numpy())
    check_matrix(qt, x.double().cpu().numpy().T)


def guarded(rows, cols):
    """An Fp4Matrix inside larger buffers of a known byte, and those buffers."""
    m = mh()
    (r, ld), (sr, sld) = m._fp4_layout(rows, cols)
    bufs = [torch.full((r * ld + 512,), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((sr * sld + 512,), 0xA5, dtype=torch.uint8, device="cuda")]
    codes = bufs[0][256:256 + r * ld].view(torch.float4_e2m1fn_x2).view(r, ld)
    scales = bufs[1][256:256 + sr * sld].view(torch.float8_e8m0fnu).view(sr, sld)
    return m.Fp4Matrix(codes, scales, (rows, cols)), bufs


@pytest.mark.parametrize("rows,cols", [(1, 1), (130, 200), (257, 513), (385, 129)])
def test_quantize_writes_its_outputs_only(rows, cols):
    x = values(rows, cols, 8)
    q, bq = guarded(rows, cols)
    t, bt = guarded(cols, rows)
    assert mh().fp4_quantize(x, forms="both", out=q, out_t=t) == (q, t)
    check_matrix(q, x.double().cpu().numpy())
    check_matrix(t, x.double().cpu().numpy().T)
    for b in bq + bt:
        assert (b[:256] == 0xA5).all() and (b[-256:] == 0xA5).all()


def test_nothing():
    for shape in ((0, 100), (100, 0), (0, 0)):
        q, qt = mh().fp4_quantize(torch.empty(shape, device="cuda"), forms="both")
        assert q.shape == shape and qt.shape == shape[::-1] and q.dequantize().shape == shape
    a, b = mh().Fp4Matrix.empty(5, 0), mh().Fp4Matrix.empty(7, 0)
    assert (mh().fp4_matmul(a, b) == 0).all()
    old = values(5, 7, 1)
    assert torch.equal(mh().fp4_matmul(a, b, out=old.clone(), accumulate=True), old)
    assert mh().fp4_matmul(mh().Fp4Matrix.empty(0, 9), mh().Fp4Matrix.empty(7, 9)).shape == (0, 7)


# ---- products --------------------------------------------------------------------
def matrix(codes, scales, shape):
    """From codes one to a byte and scale bytes, both padded."""
    m = mh()
    c = torch.from_numpy(fo.pack(codes)).cuda().view(torch.float4_e2m1fn_x2)
    return m.Fp4Matrix(c, torch.from_numpy(scales).cuda().view(torch.float8_e8m0fnu), shape)


def random_matrix(rows, cols, seed, spread=0):
    """(Fp4Matrix, its fp64 values): any codes; scales of one power per row, or spread along it."""
    rng = np.random.default_rng((seed, rows, cols))
    ld, sld = -(-cols // 256) * 256, -(-cols // 256) * 8
    codes = np.zeros((rows, ld), np.uint8)
    codes[:, :cols] = rng.integers(0, 16, (rows, cols))
    scales = np.zeros((rows, sld), np.uint8)
    nb = -(-cols // 32)
    scales[:, :nb] = 127 + rng.integers(-20, 21, (rows, 1)) + (rng.integers(-spread, spread + 1, (rows, nb)) if spread else 0)
    return matrix(codes, scales, (rows, cols)), fo.values(fo.pack(codes), scales, (rows, cols))


SIZES = [(1, 1, 1), (1, 6144, 2048), (2, 17, 129), (16, 512, 2048), (17, 130, 1000), (33, 64, 256), (64, 300, 4096),
         (65, 15, 64), (128, 128, 128), (129, 257, 769), (300, 1, 1300), (777, 1003, 501), (1024, 512, 256),
         (200, 300, 16384), (513, 2050, 640), (2100, 1100, 192), (2900, 2900, 100), (2817, 3000, 1301),
         (4096, 2048, 768), (1536, 5400, 2560), (6144, 2048, 4096), (1024, 4096, 8192)]
# each of the large tiles with 1 to 5 blocks of k, and more
SIZES += [(m, n, k) for m, n in ((1100, 1300), (2817, 3000), (3900, 4000)) for k in (200, 300, 768, 900, 1200, 1501)]


def reference(va, vb):
    return (torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda().t().contiguous())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_exact(m, n, k, dtype):
    """One scale per row: sums of whole quarters, exact whatever the order."""
    a, va = random_matrix(m, k, 1)
    b, vb = random_matrix(n, k, 2)
    want = reference(va, vb)  # below 2^24 quarters, so exact in fp64 too
    out = mh().fp4_matmul(a, b, out_dtype=DT[dtype])
    assert out.dtype == DT[dtype] and torch.equal(out, want.to(torch.float32).to(DT[dtype]))
    old = torch.full_like(out, 3.0)
    got = mh().fp4_matmul(a, b, out=old, accumulate=True)
    assert got is old and torch.equal(got, (want.float() + 3.0).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k, dtype):
    """Scales that differ along k by up to 2^20."""
    a, va = random_matrix(m, k, 3, 5)
    b, vb = random_matrix(n, k, 4, 5)
    want, p = reference(va, vb), reference(np.abs(va), np.abs(vb))
    tol = (8 * -(-k // 128) + 64) * U * p + HALF[dtype] * want.abs()
    out = mh().fp4_matmul(a, b, out_dtype=DT[dtype])
    assert ((out.double() - want).abs() <= tol).all()
    assert torch.equal(out, mh().fp4_matmul(a, b, out_dtype=DT[dtype]))
    old = torch.randn(m, n, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(DT[dtype]) * p.max().float().to(DT[dtype]) * 0.01
    old64 = old.double()
    got = mh().fp4_matmul(a, b, out=old, accumulate=True)
    want = want + old64
    assert ((got.double() - want).abs() <= tol + U * old64.abs() * 2 + HALF[dtype] * want.abs()).all()


@pytest.mark.parametrize("m,n,k", [(1, 60, 1024), (300, 520, 2048), (200, 300, 16384), (1100, 1300, 512), (2817, 3000, 512), (3900, 4000, 768)])
def test_small_sums_survive_large_products_that_cancel(m, n, k):
    """Group 0 of every row times 2^12 and group 5 its negative: what is left is the rest, exact in quarters."""
    rng = np.random.default_rng(5)
    ca, cb = rng.integers(0, 16, (m, k)).astype(np.uint8), rng.integers(0, 16, (n, k)).astype(np.uint8)
    ca[:, 160:192], cb[:, 160:192] = ca[:, :32] ^ 8, cb[:, :32]
    sld = -(-k // 256) * 8
    sa, sb = np.full((m, sld), 127, np.uint8), np.full((n, sld), 127, np.uint8)
    sa[:, [0, 5]] = 127 + 12
    want = reference(fo.values(fo.pack(ca), sa, (m, k)), fo.values(fo.pack(cb), sb, (n, k)))
    pad = lambda c: np.pad(c, ((0, 0), (0, -k % 256)))  # noqa: E731
    out = mh().fp4_matmul(matrix(pad(ca), sa, (m, k)), matrix(pad(cb), sb, (n, k)), out_dtype=torch.float32)
    # partial sums hold at most 32 * 36 * 4 * 2^12 < 2^25 quarters: one bit may go, of a step of 2 quarters
    assert ((out.double() - want).abs() <= 1.0).all()


@pytest.mark.parametrize("m,n,k", [(1, 40, 300), (70, 90, 600), (500, 520, 2000), (200, 300, 16384), (1100, 1300, 300), (2900, 2900, 100), (3900, 4000, 600)])
def test_nan_groups_stay_in_their_rows(m, n, k):
    a, va = random_matrix(m, k, 1)
    b, vb = random_matrix(n, k, 2)
    a.scales.view(torch.uint8)[m // 2, (k // 32) // 2] = 255
    b.scales.view(torch.uint8)[n // 3, -(-k // 32) - 1] = 255
    out = mh().fp4_matmul(a, b, out_dtype=torch.float32)
    want = reference(va, vb).float()
    want[m // 2] = want[:, n // 3] = float("nan")
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


def test_ends_of_the_range():
    """Products down to fp32's subnormals and up to its end."""
    m, n, k = 40, 48, 64
    rng = np.random.default_rng(7)
    codes = lambda r: np.pad(rng.integers(0, 16, (r, k)).astype(np.uint8), ((0, 0), (0, 192)))  # noqa: E731
    ca, cb = codes(m), codes(n)
    for ea, eb in ((-70, -72), (-126, -14), (-60, -60), (-127, 100), (60, 56), (127, -20), (-127, 127)):
        sa, sb = np.full((m, 8), 127 + ea, np.uint8), np.full((n, 8), 127 + eb, np.uint8)
        va, vb = fo.values(fo.pack(ca), sa, (m, k)), fo.values(fo.pack(cb), sb, (n, k))
        out = mh().fp4_matmul(matrix(ca, sa, (m, k)), matrix(cb, sb, (n, k)), out_dtype=torch.float32)
        want = reference(va, vb)
        # quarters of 2^(ea+eb); below fp32's smallest step each of the two groups may be rounded, by a step
        assert ((out.double() - want).abs() <= (0.0 if ea + eb >= -147 else 2.0 ** -148)).all(), (ea, eb)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k,ld,first", [(7, 50, 300, 51, 1), (300, 257, 600, 260, 3), (520, 1030, 512, 1031, 0), (200, 301, 16384, 303, 1), (1100, 1300, 512, 1301, 5),
                                               (2817, 3000, 300, 3007, 1), (3900, 4000, 300, 4003, 3)])
def test_output_rows_inside_wider_ones(m, n, k, ld, first, dtype):
    a, va = random_matrix(m, k, 1)
    b, vb = random_matrix(n, k, 2)
    base = torch.full(((m + 1) * ld + 16,), 7.0, device="cuda", dtype=DT[dtype])
    out = base.as_strided((m, n), (ld, 1), first)
    want = mh().fp4_matmul(a, b, out_dtype=DT[dtype])
    mh().fp4_matmul(a, b, out=out)
    assert torch.equal(out, want)
    mh().fp4_matmul(a, b, out=out, accumulate=True)
    assert torch.equal(out, (want.float() + reference(va, vb).float()).to(DT[dtype]))
    keep = torch.ones_like(base, dtype=torch.bool)
    keep.as_strided((m, n), (ld, 1), first).fill_(False)
    assert (base[keep] == 7.0).all()


def test_codes_past_32_bits():
    """The last rows of an operand of more than 2^32 bytes."""
    rows, k = 70000, 131072
    m = mh()
    big = m.Fp4Matrix(torch.zeros(rows, k // 2, dtype=torch.uint8, device="cuda").view(torch.float4_e2m1fn_x2),
                      torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu), (rows, k))
    a, va = random_matrix(3, k, 1)
    b, vb = random_matrix(3, k, 2)
    big.codes.view(torch.uint8)[-3:] = b.codes.view(torch.uint8)
    big.scales.view(torch.uint8)[-3:] = b.scales.view(torch.uint8)
    out = m.fp4_matmul(a, big, out_dtype=torch.float32)
    assert (out[:, :-3] == 0).all()
    assert torch.equal(out[:, -3:], reference(va, vb).float())
    assert torch.equal(m.fp4_matmul(big, a, out_dtype=torch.float32), out.t())


def test_quantization_past_32_bits():
    """The last rows and columns of a source of more than 2^32 bytes, codes past 2^31."""
    rows, k = 70000, 66000
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    x[-3:] = values(3, k, 1, "bf16")
    x[:, -2:] = values(rows, 2, 2, "bf16")
    q, qt = mh().fp4_quantize(x, forms="both")
    last = x[-3:].double().cpu().numpy()
    codes, scales = fo.quantize(last)
    assert np.array_equal(fo.unpack(q.codes.view(torch.uint8)[-3:].cpu().numpy()), codes)
    assert np.array_equal(q.scales.view(torch.uint8)[-3:].cpu().numpy(), scales)
    codes, scales = fo.quantize(x[:, -2:].double().cpu().numpy().T)
    assert np.array_equal(fo.unpack(qt.codes.view(torch.uint8)[-2:].cpu().numpy()), codes)
    assert np.array_equal(qt.scales.view(torch.uint8)[-2:].cpu().numpy(), scales)
    v = q.dequantize(torch.bfloat16)
    assert np.array_equal(v[-3:].double().cpu().numpy(), fo.values(*(t.view(torch.uint8)[-3:].cpu().numpy() for t in (q.codes, q.scales)), (3, k)))
    assert not v[:-3, :-32].any()


def test_python_refuses():
    m = mh()
    a, b = m.Fp4Matrix.empty(3, 100), m.Fp4Matrix.empty(4, 100)
    x = values(3, 100, 1)
    for call in (lambda: m.fp4_matmul(a, m.Fp4Matrix.empty(4, 99)), lambda: m.fp4_matmul(a, b, accumulate=True),
                 lambda: m.fp4_matmul(a, b, out=torch.empty(4, 3, device="cuda")), lambda: m.fp4_quantize(x, forms="x"),
                 lambda: m.fp4_quantize(x, out_t=b), lambda: m.fp4_quantize(x, out=b), lambda: m.fp4_quantize(x.t()),
                 lambda: m.fp4_matmul(a, b, out=torch.empty(3, 4))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: m.fp4_matmul(a, b, out_dtype=torch.half), lambda: m.fp4_quantize(x.half()), lambda: m.fp4_quantize(x, out=x),
                 lambda: m.fp4_matmul(a, m.Fp8Matrix.empty(4, 100)), lambda: a.dequantize(torch.half),
                 lambda: m.fp4_matmul(a, b, out=torch.empty(3, 4, device="cuda"), out_dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            call()
    c = copy.deepcopy(a)
    assert c.desc.codes == c.codes.data_ptr() != a.codes.data_ptr()


def test_captured_graph_and_other_stream():
    x, w = values(300, 2048, 1, "bf16"), values(520, 2048, 2)
    dy = values(300, 520, 3, "bf16")
    # k split over workgroups: a workspace of its own in the graph
    xl, wl = values(100, 16384, 5, "bf16"), values(200, 16384, 6, "bf16")
    g = torch.zeros(520, 2048, device="cuda")

    def run(g):
        q, qt = mh().fp4_quantize(x, forms="both")
        d, dt = mh().fp4_quantize(dy, forms="both")
        p, pt = mh().fp4_quantize(w, forms="both")
        y = mh().fp4_matmul(q, p)
        dx = mh().fp4_matmul(d, pt)
        mh().fp4_matmul(dt, qt, out=g)
        mh().fp4_matmul(dt, qt, out=g, accumulate=True)
        long = mh().fp4_matmul(mh().fp4_quantize(xl)[0], mh().fp4_quantize(wl)[0], out_dtype=torch.float32)
        return [y, dx, long, q.dequantize()]

    run(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(g)
    side = torch.cuda.Stream()
    for i in range(3):
        x.copy_(values(300, 2048, 10 + i, "bf16"))
        xl.copy_(values(100, 16384, 20 + i, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held] + [g.clone()]
        other = torch.empty_like(g)
        want = run(other) + [other]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            third = torch.empty_like(g)
            again = run(third) + [third]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(again, want))
