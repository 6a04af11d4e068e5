"""Block-scaled 8-bit operators without a GPU: the oracle against independent
values, the layout functions, and every refusal of the C entry points (fake
addresses, never dereferenced: each call is rejected before device work)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import orthogonalized_updates_amd as mh
from oracle import fp8_oracle as fo

A = 1 << 32  # fake device addresses, far apart


# ---- oracle ------------------------------------------------------------------
def test_grid_is_torchs_e4m3():
    torch = pytest.importorskip("torch")
    c = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(c.view(torch.float8_e4m3fn).double().numpy(), fo.grid())


def test_encode_rounds_to_nearest_even():
    torch = pytest.importorskip("torch")
    g = fo.grid()
    mid = (g[1:] + g[:-1]) / 2
    v = np.concatenate([g, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9)])
    v = np.concatenate([v, -v])
    # fp32 holds the grid and its midpoints, not their fp64 neighbours
    exact = v == v.astype(np.float32)
    want = torch.from_numpy(v[exact].astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fo.encode(v[exact]), want)
    n = len(g) + len(mid)
    assert np.array_equal(fo.encode(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(fo.encode(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert exact.sum() >= 2 * n


@pytest.mark.parametrize("a,e", [(448.0, 0), (np.nextafter(np.float32(448), np.float32(1e9)), 1), (1.75, -8),
                                 (1.8, -7), (0.0, -126), (1e-45, -126), (3.4e38, 120), (2.0 ** -118, -126),
                                 (449 * 2.0 ** -126, -125)])
def test_scale_is_the_smallest_that_holds_the_block(a, e):
    x = np.zeros((1, 200))
    x[0, 5] = -a
    codes, scales = fo.quantize(x)
    assert codes.shape == (1, 256) and scales.shape == (1, 4)
    assert scales[0].tolist() == [e + 127, 1, 0, 0]
    assert not codes[0, 200:].any()


def test_values_inverts_exact_inputs():
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 126, (130, 128), dtype=np.uint8)
    codes[:, 0] = 126  # every block has a full-scale entry, so scales come back
    v = fo.decode(codes) * 2.0 ** 5
    for block in ("rows", "tiles"):
        q, s = fo.quantize(v, block)
        assert np.array_equal(q, codes) and set(s[:, 0]) == {132}
        assert np.array_equal(fo.values(q, s, v.shape, block), v)


# ---- layout -------------------------------------------------------------------
@pytest.mark.parametrize("cols,ld,sld", [(0, 0, 0), (1, 128, 4), (128, 128, 4), (129, 256, 4), (512, 512, 4),
                                         (513, 640, 8), (1 << 24, 1 << 24, 1 << 17), (-1, 0, 0),
                                         ((1 << 24) + 1, 0, 0)])
def test_pitches(cols, ld, sld):
    assert mh.lib.muonh_fp8_ld(cols) == ld
    assert mh.lib.muonh_fp8_scale_ld(cols) == sld


def test_scale_rows():
    assert mh.lib.muonh_fp8_scale_rows(129, mh.MUONH_FP8_ROWS) == 129
    assert mh.lib.muonh_fp8_scale_rows(129, mh.MUONH_FP8_TILES) == 2
    assert mh.lib.muonh_fp8_scale_rows(0, mh.MUONH_FP8_TILES) == 0
    assert mh.lib.muonh_fp8_scale_rows(129, 2) == 0
    assert mh.lib.muonh_fp8_scale_rows(-1, 0) == 0


def test_constants_match_the_header():
    text = mh.HEADER_PATH.read_text()
    assert "MUONH_FP8_ROWS = 0, MUONH_FP8_TILES = 1" in text
    assert "MUONH_DT_FP32 = 0, MUONH_DT_BF16 = 1" in text
    assert "#define MUONH_MAX_FP8_DIM (1 << 24)" in text and mh.MUONH_MAX_FP8_DIM == 1 << 24


# ---- refusals -------------------------------------------------------------------
def _quantize(src=A, dtype=0, rows=100, cols=200, ld=200, block=0, codes=2 * A, scales=3 * A, codes_t=None,
              scales_t=None):
    return mh.lib.muonh_fp8_quantize(src, dtype, rows, cols, ld, block, codes, scales, codes_t, scales_t, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), mh.MUONH_EINVAL),
    (dict(block=2), mh.MUONH_EINVAL),
    (dict(rows=-1), mh.MUONH_ESHAPE),
    (dict(cols=(1 << 24) + 1, ld=1 << 25), mh.MUONH_ESHAPE),
    (dict(ld=199), mh.MUONH_EINVAL),
    (dict(ld=(1 << 36) + 1), mh.MUONH_EINVAL),
    (dict(src=None), mh.MUONH_EINVAL),
    (dict(src=A + 2), mh.MUONH_EINVAL),                      # fp32 source off its alignment
    (dict(codes=None), mh.MUONH_EINVAL),                     # scales without codes
    (dict(codes=None, scales=None), mh.MUONH_EINVAL),        # no output
    (dict(codes_t=4 * A), mh.MUONH_EINVAL),                  # half a pair
    (dict(codes=2 * A + 8), mh.MUONH_EINVAL),
    (dict(scales=3 * A + 2), mh.MUONH_EINVAL),
    (dict(rows=1 << 24, cols=1 << 14, ld=1 << 14), mh.MUONH_ESHAPE),  # 2^24 tiles
    (dict(codes=A), mh.MUONH_EALIAS),
    (dict(codes=A + 100 * 200 * 4 - 16), mh.MUONH_EALIAS),   # the source's last bytes
    (dict(scales=2 * A + 99 * 256), mh.MUONH_EALIAS),        # the codes' last row
    (dict(codes_t=2 * A, scales_t=5 * A), mh.MUONH_EALIAS),
])
def test_quantize_refuses(kw, code):
    assert _quantize(**kw) == code
    assert mh.lib.muonh_last_error()


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0, ld=0), dict(rows=0, src=None, codes=None, scales=None)])
def test_quantize_of_nothing_is_a_no_op(kw):
    assert _quantize(**kw) == mh.MUONH_OK


def test_weights_refuses():
    p = mh.Plan([(8, 8, 1)])
    f = mh.lib.muonh_fp8_weights
    assert f(None, A, A, A, A, A, None) == mh.MUONH_EINVAL
    for i in range(3):
        args = [A, A, A]
        args[i] = None
        assert f(p.handle, *args, A, A, None) == mh.MUONH_EINVAL
    assert f(p.handle, A, A, A, A, None, None) == mh.MUONH_EINVAL
    assert f(p.handle, A, A, A, None, A, None) == mh.MUONH_EINVAL
    # thin matrices: 33024 of 512 tiles each, past one launch
    big = mh.Plan([(8, 8, 1), (1, 65536, 33024)])
    assert f(big.handle, A, A, A, A, A, None) == mh.MUONH_ESHAPE


def _desc(codes=A, scales=2 * A, rows=100, cols=200, block=0):
    return mh.Fp8Desc(codes, scales, rows, cols, block)


def _matmul(a=None, b=None, out=5 * A, dt=1, ld=None, acc=0, ws=None, nbytes=0):
    a = _desc() if a is None else a
    b = _desc(3 * A, 4 * A, 300) if b is None else b
    ld = b.rows if ld is None else ld
    return mh.lib.muonh_fp8_matmul(ctypes.byref(a), ctypes.byref(b), out, dt, ld, acc, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(a=_desc(rows=-1)), mh.MUONH_ESHAPE),
    (dict(b=_desc(cols=(1 << 24) + 1)), mh.MUONH_ESHAPE),
    (dict(a=_desc(block=2)), mh.MUONH_EINVAL),
    (dict(a=_desc(codes=None)), mh.MUONH_EINVAL),
    (dict(b=_desc(scales=None)), mh.MUONH_EINVAL),
    (dict(a=_desc(codes=A + 8)), mh.MUONH_EINVAL),
    (dict(b=_desc(scales=2 * A + 1)), mh.MUONH_EINVAL),
    (dict(a=_desc(cols=201)), mh.MUONH_ESHAPE),
    (dict(dt=2), mh.MUONH_EINVAL),
    (dict(ld=299), mh.MUONH_EINVAL),
    (dict(ld=(1 << 36) + 1), mh.MUONH_EINVAL),
    (dict(out=None), mh.MUONH_EINVAL),
    (dict(out=5 * A + 1), mh.MUONH_EINVAL),
    (dict(out=5 * A + 2, dt=0), mh.MUONH_EINVAL),
    (dict(a=_desc(rows=1 << 24), b=_desc(rows=1 << 11), out=9 * A), mh.MUONH_ESHAPE),
    (dict(out=A), mh.MUONH_EALIAS),                               # a's codes
    (dict(out=3 * A + 299 * 256), mh.MUONH_EALIAS),               # b's last row
    (dict(out=2 * A - 100 * 300 * 2 + 2), mh.MUONH_EALIAS),       # ends inside a's scales
])
def test_matmul_refuses(kw, code):
    assert _matmul(**kw) == code
    assert mh.lib.muonh_last_error()


def test_matmul_refuses_null_operands():
    d = _desc()
    assert mh.lib.muonh_fp8_matmul(None, ctypes.byref(d), A, 1, 100, 0, None, 0, None) == mh.MUONH_EINVAL
    assert mh.lib.muonh_fp8_matmul(ctypes.byref(d), None, A, 1, 100, 0, None, 0, None) == mh.MUONH_EINVAL


def test_matmul_workspace_is_checked():
    a, b = _desc(rows=200, cols=8192), _desc(3 * A, 4 * A, 300, 8192)
    for dt in (0, 1):
        need = mh.lib.muonh_fp8_matmul_workspace_bytes(200, 300, 8192, dt)
        assert need > 0
        assert _matmul(a, b, dt=dt) == mh.MUONH_EWORKSPACE
        assert _matmul(a, b, dt=dt, ws=6 * A + 16, nbytes=need) == mh.MUONH_EWORKSPACE
        assert _matmul(a, b, dt=dt, ws=6 * A, nbytes=need - 1) == mh.MUONH_EWORKSPACE
        assert "needs" in mh.lib.muonh_last_error().decode()
        assert _matmul(a, b, dt=dt, ws=5 * A, nbytes=need) == mh.MUONH_EALIAS
        assert _matmul(a, b, dt=dt, ws=3 * A, nbytes=need) == mh.MUONH_EALIAS
    for m, n, k in ((-1, 4, 4), (0, 5, 5), (5, 0, 5), (1 << 25, 4, 4), (8192, 8192, 8192)):
        assert mh.lib.muonh_fp8_matmul_workspace_bytes(m, n, k, 0) == 0


def test_matmul_of_nothing_is_a_no_op():
    assert _matmul(a=_desc(rows=0)) == mh.MUONH_OK
    assert _matmul(b=_desc(None, None, 0), ld=0, out=None) == mh.MUONH_OK


# ---- binding --------------------------------------------------------------------
def test_binding_refuses_without_a_gpu():
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError):
        mh.fp8_quantize([[1.0]])
    with pytest.raises(TypeError):
        mh.fp8_quantize(torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        mh.fp8_quantize(torch.zeros(4, 4))
    with pytest.raises(TypeError):
        mh.fp8_matmul(torch.zeros(4, 4), torch.zeros(4, 4))
    codes = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    scales = torch.zeros(4, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    with pytest.raises(ValueError, match="GPU"):
        mh.Fp8Matrix(codes, scales, (4, 100))
    with pytest.raises(ValueError, match="block"):
        mh.Fp8Matrix(codes, scales, (4, 100), "columns")
    with pytest.raises(ValueError, match="contiguous"):
        mh.Fp8Matrix(codes, scales, (4, 129))
    with pytest.raises(TypeError, match="scales"):
        mh.Fp8Matrix(codes, scales.view(torch.uint8), (4, 100))
    with pytest.raises(ValueError, match="shape"):
        mh.Fp8Matrix(codes, scales, (4, -1))


@pytest.mark.parametrize("device,on", [(0, "cuda:0"), (3, "cuda:3"), (None, "cuda"), ("cuda:1", "cuda:1")])
def test_empty_takes_the_device_asked_for(monkeypatch, device, on):
    """Number 0 is the first GPU, not "no device given"."""
    torch = pytest.importorskip("torch")
    asked, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda s, dtype, device: asked.append(device) or empty(s, dtype=dtype))
    mh.Fp8Matrix.empty(4, 100, device=device)
    assert asked == [torch.device(on)] * 2


def test_matmul_takes_fast_for_bf16_results_only():
    assert f"MUONH_FP8_FAST = {mh.MUONH_FP8_FAST}" in mh.HEADER_PATH.read_text()
    fast = mh.MUONH_FP8_FAST
    for dt in (mh.MUONH_DT_FP32 | fast, fast | 2, 2 * fast | mh.MUONH_DT_BF16, -1):
        assert _matmul(dt=dt) == mh.MUONH_EINVAL
    assert _matmul(dt=mh.MUONH_DT_BF16 | fast, ld=299) == mh.MUONH_EINVAL  # past the type's check
    assert "out_ld" in mh.lib.muonh_last_error().decode()
    need = mh.lib.muonh_fp8_matmul_workspace_bytes(200, 300, 8192, mh.MUONH_DT_BF16 | fast)
    a, b = _desc(rows=200, cols=8192), _desc(3 * A, 4 * A, 300, 8192)
    assert need > 0 and _matmul(a, b, dt=mh.MUONH_DT_BF16 | fast, ws=6 * A, nbytes=need - 1) == mh.MUONH_EWORKSPACE
