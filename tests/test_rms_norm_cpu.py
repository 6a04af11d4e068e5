"""RMS norm without a GPU: the oracle against differences, every refusal of the C
entry points (fake addresses, never dereferenced: each call is rejected before
device work) and of the Python functions."""
from __future__ import annotations

import numpy as np
import pytest

import orthogonalized_updates_amd as mh
from oracle import norm_oracle as no

A = 1 << 32  # fake device addresses, far apart
BIG = (1 << 24) + 1


def test_oracle_gradient_against_differences():
    """Central differences of fp64 sums: error about step^2 * (third derivative), 1e-9 here."""
    rng = np.random.default_rng(1)
    h, w, t = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    eps, step = 1e-2, 1e-5
    f = lambda h, w: float(np.sum(t * no.forward(h, w, eps)[0]))  # noqa: E731
    dh, dw = no.backward(t, h, w, no.forward(h, w, eps)[1])
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = step
        assert abs((f(h + d, w) - f(h - d, w)) / (2 * step) - dh[i]) < 1e-8
    for j in range(7):
        d = np.zeros_like(w)
        d[j] = step
        assert abs((f(h, w + d) - f(h, w - d)) / (2 * step) - dw[j]) < 1e-8


def _forward(x=A, dt=0, rows=100, cols=200, ld=200, res=2 * A, hdt=0, rld=200, h=3 * A, hld=200, w=4 * A, eps=1e-6,
             rstd=5 * A, y=6 * A, ydt=0, yld=200, codes=None, scales=None, codes_t=None, scales_t=None):
    return mh.lib.muonh_rms_norm(x, dt, rows, cols, ld, res, hdt, rld, h, hld, w, eps, rstd, y, ydt, yld, codes, scales,
                                 codes_t, scales_t, None)


F8 = dict(y=None, codes=7 * A, scales=8 * A)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), mh.MUONH_EINVAL), (dict(hdt=-1), mh.MUONH_EINVAL), (dict(ydt=256), mh.MUONH_EINVAL),
    (dict(rows=-1), mh.MUONH_ESHAPE), (dict(cols=0), mh.MUONH_ESHAPE), (dict(rows=BIG), mh.MUONH_ESHAPE),
    (dict(cols=BIG, ld=BIG, rld=BIG, hld=BIG, yld=BIG), mh.MUONH_ESHAPE),
    (dict(eps=-1e-9), mh.MUONH_EINVAL), (dict(eps=float("nan")), mh.MUONH_EINVAL), (dict(eps=float("inf")), mh.MUONH_EINVAL),
    (dict(x=None), mh.MUONH_EINVAL), (dict(w=None), mh.MUONH_EINVAL), (dict(rstd=None), mh.MUONH_EINVAL),
    (dict(h=None), mh.MUONH_EINVAL), (dict(res=None), mh.MUONH_EINVAL),          # one of residual and h
    (dict(ld=199), mh.MUONH_EINVAL), (dict(rld=199), mh.MUONH_EINVAL), (dict(hld=199), mh.MUONH_EINVAL),
    (dict(yld=199), mh.MUONH_EINVAL), (dict(ld=(1 << 36) + 1), mh.MUONH_EINVAL),
    (dict(x=A + 2), mh.MUONH_EINVAL), (dict(dt=1, x=A + 1), mh.MUONH_EINVAL), (dict(w=4 * A + 2), mh.MUONH_EINVAL),
    (dict(rstd=5 * A + 1), mh.MUONH_EINVAL), (dict(y=6 * A + 2), mh.MUONH_EINVAL), (dict(h=3 * A + 1), mh.MUONH_EINVAL),
    (dict(y=None), mh.MUONH_EINVAL),                                             # no output
    (dict(codes=7 * A, scales=8 * A), mh.MUONH_EINVAL),                          # both kinds
    (dict(F8, scales=None), mh.MUONH_EINVAL), (dict(F8, codes_t=9 * A), mh.MUONH_EINVAL),
    (dict(F8, codes=7 * A + 8), mh.MUONH_EINVAL), (dict(F8, scales=8 * A + 2), mh.MUONH_EINVAL),
    (dict(F8, rows=1 << 24, cols=1 << 14, ld=1 << 14, rld=1 << 14, hld=1 << 14, x=A, res=400 * A, h=800 * A,
          codes=1200 * A, scales=1600 * A, codes_t=2000 * A, scales_t=2400 * A), mh.MUONH_ESHAPE),  # 2^24 tiles
    (dict(h=2 * A, hld=300), mh.MUONH_EALIAS),                                   # in place, other pitch
    (dict(h=A, hdt=1), mh.MUONH_EALIAS),                                         # in place, other type
    (dict(h=2 * A + 4), mh.MUONH_EALIAS), (dict(y=A), mh.MUONH_EALIAS), (dict(y=3 * A + 99 * 800), mh.MUONH_EALIAS),
    (dict(rstd=4 * A + 796), mh.MUONH_EALIAS), (dict(rstd=A + 400), mh.MUONH_EALIAS),
    (dict(F8, codes=A), mh.MUONH_EALIAS), (dict(F8, scales=7 * A + 99 * 256), mh.MUONH_EALIAS),
    (dict(F8, codes_t=7 * A, scales_t=9 * A), mh.MUONH_EALIAS),
])
def test_forward_refuses(kw, code):
    assert _forward(**kw) == code
    assert mh.lib.muonh_last_error()


@pytest.mark.parametrize("apart,meets", [(800, False), (4000, False), (8800, False), (796, True), (4, True), (9600, True), (8804, True),
                                         (-800, False), (-796, True), (-8800, False), (-9600, True)])
def test_rows_may_lie_between_each_other(apart, meets):
    """dh's 200 floats per row in the same rows of 2400 floats as dy's, `apart` bytes on."""
    f = mh.lib.muonh_rms_norm_backward
    dh = A + (1 << 20) + apart
    got = f(A + (1 << 20), 0, 2400, 9 * A, 0, 100, 200, 200, 3 * A, 4 * A, None, 0, dh, 2400, 7 * A if meets else 4 * A + 4, 0, 8 * A, 1 << 40, None)
    # the accepted ones go on to the next check, which refuses dweight for overlapping rstd
    assert got == mh.MUONH_EALIAS
    assert (b"dh overlaps dy" in mh.lib.muonh_last_error()) == meets


def test_forward_of_no_rows_is_a_no_op():
    assert _forward(rows=0, x=None, res=None, h=None, y=None, w=None, rstd=None) == mh.MUONH_OK


def _backward(dy=A, ddt=0, dld=200, h=2 * A, hdt=0, rows=100, cols=200, hld=200, w=3 * A, rstd=4 * A, res=5 * A, rld=200,
              dh=6 * A, old=200, dw=7 * A, acc=0, ws=8 * A, nbytes=1 << 40):
    return mh.lib.muonh_rms_norm_backward(dy, ddt, dld, h, hdt, rows, cols, hld, w, rstd, res, rld, dh, old, dw, acc, ws,
                                          nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ddt=2), mh.MUONH_EINVAL), (dict(hdt=2), mh.MUONH_EINVAL), (dict(rows=-1), mh.MUONH_ESHAPE),
    (dict(cols=0), mh.MUONH_ESHAPE), (dict(rows=BIG), mh.MUONH_ESHAPE),
    (dict(dy=None), mh.MUONH_EINVAL), (dict(h=None), mh.MUONH_EINVAL), (dict(w=None), mh.MUONH_EINVAL),
    (dict(rstd=None), mh.MUONH_EINVAL), (dict(dh=None), mh.MUONH_EINVAL), (dict(dw=None), mh.MUONH_EINVAL),
    (dict(dld=199), mh.MUONH_EINVAL), (dict(hld=199), mh.MUONH_EINVAL), (dict(rld=199), mh.MUONH_EINVAL),
    (dict(old=199), mh.MUONH_EINVAL), (dict(dy=A + 2), mh.MUONH_EINVAL), (dict(dw=7 * A + 2), mh.MUONH_EINVAL),
    (dict(ws=None), mh.MUONH_EWORKSPACE), (dict(ws=8 * A + 128), mh.MUONH_EWORKSPACE),
    (dict(nbytes=25 * 200 * 4 - 1), mh.MUONH_EWORKSPACE),
    (dict(dh=2 * A), mh.MUONH_EALIAS),                       # h is read after the first store
    (dict(dh=A, hdt=1, h=2 * A), mh.MUONH_EALIAS),           # in dy's place, other type
    (dict(dh=5 * A, old=201), mh.MUONH_EALIAS), (dict(dw=3 * A), mh.MUONH_EALIAS), (dict(dw=6 * A + 400), mh.MUONH_EALIAS),
    (dict(ws=2 * A), mh.MUONH_EALIAS), (dict(ws=7 * A), mh.MUONH_EALIAS),
])
def test_backward_refuses(kw, code):
    assert _backward(**kw) == code
    assert mh.lib.muonh_last_error()


def test_backward_workspace():
    f = mh.lib.muonh_rms_norm_backward_workspace_bytes
    assert f(0, 5) == f(5, 0) == f(-1, 5) == f(5, BIG) == 0
    assert f(100, 200) == 25 * 200 * 4              # 4 rows at a time
    assert f(1, 2048) == 2048 * 4
    assert f(1 << 20, 2048) == 512 * 2048 * 4
    assert f(10, 16384) == 10 * 16384 * 4
    assert f(10, 16385) == (10 * 16385 + 10) * 4    # and the rows' means
    assert f(5, 1 << 24) == (5 * (1 << 24) + 5) * 4


def test_python_refuses():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 4), torch.ones(4)
    for call in (lambda: mh.rms_norm(x, w), lambda: mh.rms_norm_fp8(x, w), lambda: mh.rms_norm_backward(x, x, w, torch.ones(2))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        mh.rms_norm([1.0], w)
    with pytest.raises(TypeError):
        mh.rms_norm(x.half(), w)
    with pytest.raises(ValueError, match="forms"):
        mh.rms_norm_fp8(x, w, forms="neither")
