"""Microscaled 4-bit operators without a GPU: the oracle against independent
values, the layout functions, every refusal of the C entry points (fake addresses,
never dereferenced) and of the Python functions."""
from __future__ import annotations

import copy
import ctypes

import numpy as np
import pytest

import orthogonalized_updates_amd as mh
from oracle import fp4_oracle as fo

A = 1 << 32  # fake device addresses, far apart


def test_grid_from_the_bits():
    """Sign, exponent with bias 1, one mantissa bit; exponent 0 without the leading one."""
    for code in range(16):
        e, m = code >> 1 & 3, code & 1
        v = (1 + m / 2) * 2.0 ** (e - 1) if e else m / 2
        assert fo.decode(np.array([code], np.uint8))[0] == (-v if code & 8 else v)


def test_encode_rounds_to_nearest_even():
    g = fo.GRID
    mid = (g[1:] + g[:-1]) / 2
    assert fo.encode(g).tolist() == list(range(8)) and fo.encode(-g).tolist() == list(range(8, 16))
    assert fo.encode(mid).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert fo.encode(np.nextafter(mid, 0)).tolist() == list(range(7))
    assert fo.encode(np.nextafter(mid, 9)).tolist() == list(range(1, 8))


@pytest.mark.parametrize("a,e", [(6.0, 0), (np.nextafter(np.float32(6), np.float32(9)), 1), (3.0, -1), (4.0, 0), (3.1, 0), (0.0, -126),
                                 (1e-45, -126), (3.4e38, 126), (6 * 2.0 ** -126, -126), (6.5 * 2.0 ** -126, -125)])
def test_scale_is_the_smallest_that_holds_the_group(a, e):
    x = np.zeros((1, 70))
    x[0, 35] = -a
    codes, scales = fo.quantize(x)
    assert codes.shape == (1, 256) and scales.shape == (1, 8)
    assert scales[0, :4].tolist() == [1, e + 127, 1, 0] and not scales[0, 4:].any() and not codes[0, 70:].any()
    x[0, 64] = np.nan
    codes, scales = fo.quantize(x)
    assert scales[0, :3].tolist() == [1, e + 127, 255] and not codes[0, 64:].any()


def test_pack_and_values():
    codes = np.random.default_rng(1).integers(0, 16, (3, 256), dtype=np.uint8)
    assert np.array_equal(fo.unpack(fo.pack(codes)), codes) and fo.pack(codes)[0, 0] == codes[0, 0] + 16 * codes[0, 1]
    s = np.full((3, 8), 130, np.uint8)
    assert np.array_equal(fo.values(fo.pack(codes), s, (3, 200)), 8 * fo.decode(codes[:, :200]))


@pytest.mark.parametrize("cols,ld,sld", [(0, 0, 0), (1, 128, 8), (256, 128, 8), (257, 256, 16), (512, 256, 16), (513, 384, 24),
                                         (1 << 24, 1 << 23, 1 << 19), (-1, 0, 0), ((1 << 24) + 1, 0, 0)])
def test_pitches(cols, ld, sld):
    assert mh.lib.muonh_fp4_ld(cols) == ld
    assert mh.lib.muonh_fp4_scale_ld(cols) == sld
    if 0 <= cols <= 1 << 24:
        assert mh._fp4_layout(3, cols) == ((3, ld), (3, sld))


def _quantize(src=A, dtype=0, rows=100, cols=200, ld=200, codes=2 * A, scales=3 * A, codes_t=None, scales_t=None):
    return mh.lib.muonh_fp4_quantize(src, dtype, rows, cols, ld, codes, scales, codes_t, scales_t, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), mh.MUONH_EINVAL), (dict(rows=-1), mh.MUONH_ESHAPE), (dict(cols=(1 << 24) + 1, ld=1 << 25), mh.MUONH_ESHAPE),
    (dict(ld=199), mh.MUONH_EINVAL), (dict(ld=(1 << 36) + 1), mh.MUONH_EINVAL), (dict(src=None), mh.MUONH_EINVAL),
    (dict(src=A + 2), mh.MUONH_EINVAL), (dict(codes=None), mh.MUONH_EINVAL), (dict(codes=None, scales=None), mh.MUONH_EINVAL),
    (dict(codes_t=4 * A), mh.MUONH_EINVAL), (dict(codes=2 * A + 8), mh.MUONH_EINVAL), (dict(scales=3 * A + 4), mh.MUONH_EINVAL),
    (dict(rows=1 << 24, cols=1 << 14, ld=1 << 14, codes=400 * A, scales=800 * A), mh.MUONH_ESHAPE),
    (dict(codes=A), mh.MUONH_EALIAS), (dict(codes=A + 79984), mh.MUONH_EALIAS), (dict(scales=2 * A + 99 * 128), mh.MUONH_EALIAS),
    (dict(codes_t=2 * A, scales_t=5 * A), mh.MUONH_EALIAS),
])
def test_quantize_refuses(kw, code):
    assert _quantize(**kw) == code
    assert mh.lib.muonh_last_error()


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0, ld=0), dict(rows=0, src=None, codes=None, scales=None)])
def test_quantize_of_nothing_is_a_no_op(kw):
    assert _quantize(**kw) == mh.MUONH_OK


def _matrix(codes=A, scales=2 * A, rows=100, cols=200):
    return mh.Fp4Desc(codes, scales, rows, cols)


def test_dequantize_refuses():
    f = mh.lib.muonh_fp4_dequantize
    m = _matrix()
    assert f(None, 3 * A, 0, 200, None) == mh.MUONH_EINVAL
    assert f(ctypes.byref(m), None, 0, 200, None) == mh.MUONH_EINVAL
    assert f(ctypes.byref(m), 3 * A, 2, 200, None) == mh.MUONH_EINVAL
    assert f(ctypes.byref(m), 3 * A, 0, 199, None) == mh.MUONH_EINVAL
    assert f(ctypes.byref(m), 3 * A + 2, 0, 200, None) == mh.MUONH_EINVAL
    assert f(ctypes.byref(m), A, 0, 200, None) == mh.MUONH_EALIAS
    assert f(ctypes.byref(m), 2 * A + 796, 0, 200, None) == mh.MUONH_EALIAS
    assert f(ctypes.byref(_matrix(codes=None)), 3 * A, 0, 200, None) == mh.MUONH_EINVAL
    assert f(ctypes.byref(_matrix(rows=-1)), 3 * A, 0, 200, None) == mh.MUONH_ESHAPE
    assert f(ctypes.byref(_matrix(rows=0)), None, 0, 200, None) == mh.MUONH_OK


def _matmul(a=None, b=None, out=9 * A, dt=0, ld=300, acc=0, ws=None, size=0):
    a = a or _matrix()
    b = b or _matrix(4 * A, 5 * A, 300)
    return mh.lib.muonh_fp4_matmul(ctypes.byref(a), ctypes.byref(b), out, dt, ld, acc, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(a=_matrix(codes=None)), mh.MUONH_EINVAL), (dict(b=_matrix(scales=None)), mh.MUONH_EINVAL),
    (dict(a=_matrix(codes=A + 8)), mh.MUONH_EINVAL), (dict(a=_matrix(scales=2 * A + 4)), mh.MUONH_EINVAL),
    (dict(a=_matrix(rows=-1)), mh.MUONH_ESHAPE), (dict(a=_matrix(cols=(1 << 24) + 1)), mh.MUONH_ESHAPE),
    (dict(a=_matrix(cols=201)), mh.MUONH_ESHAPE), (dict(dt=2), mh.MUONH_EINVAL), (dict(dt=257), mh.MUONH_EINVAL),
    (dict(ld=299), mh.MUONH_EINVAL), (dict(ld=(1 << 36) + 1), mh.MUONH_EINVAL), (dict(out=None), mh.MUONH_EINVAL),
    (dict(out=9 * A + 2), mh.MUONH_EINVAL), (dict(out=9 * A + 1, dt=1), mh.MUONH_EINVAL),
    (dict(a=_matrix(rows=1 << 18), b=_matrix(400 * A, 500 * A, 1 << 18), ld=1 << 18, out=900 * A), mh.MUONH_ESHAPE),
    (dict(out=A), mh.MUONH_EALIAS), (dict(out=2 * A - 4), mh.MUONH_EALIAS), (dict(out=4 * A + 299 * 128), mh.MUONH_EALIAS),
    (dict(out=5 * A), mh.MUONH_EALIAS),
])
def test_matmul_refuses(kw, code):
    assert _matmul(**kw) == code
    assert mh.lib.muonh_last_error()


def test_matmul_null_and_workspace():
    m = _matrix()
    f = mh.lib.muonh_fp4_matmul
    assert f(None, ctypes.byref(m), 9 * A, 0, 100, 0, None, 0, None) == mh.MUONH_EINVAL
    assert f(ctypes.byref(m), None, 9 * A, 0, 100, 0, None, 0, None) == mh.MUONH_EINVAL
    size = mh.lib.muonh_fp4_matmul_workspace_bytes(200, 300, 16384)
    assert size > 0
    a, b = _matrix(A, 2 * A, 200, 16384), _matrix(4 * A, 5 * A, 300, 16384)
    assert _matmul(a, b, ws=None, size=size) == mh.MUONH_EWORKSPACE
    assert _matmul(a, b, ws=7 * A + 128, size=size) == mh.MUONH_EWORKSPACE
    assert _matmul(a, b, ws=7 * A, size=size - 1) == mh.MUONH_EWORKSPACE
    assert _matmul(a, b, ws=9 * A + 256, size=size) == mh.MUONH_EALIAS
    assert _matmul(a, b, ws=5 * A, size=size) == mh.MUONH_EALIAS
    assert mh.lib.muonh_fp4_matmul_workspace_bytes(0, 3, 5) == mh.lib.muonh_fp4_matmul_workspace_bytes(3, 5, -1) == 0
    assert _matmul(_matrix(rows=0), out=None) == mh.MUONH_OK
    assert _matmul(b=_matrix(4 * A, 5 * A, 0), out=None, ld=0) == mh.MUONH_OK


def test_python_refuses():
    torch = pytest.importorskip("torch")
    codes = torch.zeros(3, 128, dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    scales = torch.zeros(3, 8, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    with pytest.raises(ValueError, match="GPU"):
        mh.Fp4Matrix(codes, scales, (3, 200))
    with pytest.raises(ValueError, match="GPU"):
        mh.Fp4Matrix.empty(3, 200, device="cpu")
    with pytest.raises(ValueError):
        mh.Fp4Matrix(codes, scales, (3, 300))
    with pytest.raises(TypeError):
        mh.Fp4Matrix(codes.view(torch.uint8), scales, (3, 200))
    with pytest.raises(ValueError):
        mh.Fp4Matrix.empty(3, -1)
    with pytest.raises(ValueError, match="GPU"):
        mh.fp4_quantize(torch.zeros(3, 4))
    with pytest.raises(TypeError):
        mh.fp4_matmul(torch.zeros(3, 4), torch.zeros(3, 4))
    m = mh.Fp4Matrix.__new__(mh.Fp4Matrix)
    m._set(codes, scales, (3, 200))
    for name in ("codes", "scales", "shape", "desc", "device"):
        with pytest.raises(AttributeError, match="Fp4Matrix"):
            setattr(m, name, None)
        with pytest.raises(AttributeError):
            delattr(m, name)
    assert m.__reduce__()[0] is mh.Fp4Matrix and copy.copy(m.shape) == (3, 200)
    with pytest.raises(TypeError):
        mh.fp4_matmul(m, "b")
    codes.data = torch.zeros(3, 128, dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    with pytest.raises(ValueError, match="moved"):
        mh.fp4_matmul(m, m)
