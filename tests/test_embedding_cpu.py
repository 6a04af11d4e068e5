"""Embedding without a GPU: the oracle against index operations of torch, every
refusal of the C entry points (fake addresses, never dereferenced) and of the
Python functions."""
from __future__ import annotations

import numpy as np
import pytest

import orthogonalized_updates_amd as mh
from oracle import embedding_oracle as eo

A = 1 << 36  # fake device addresses, far apart
BIG = (1 << 24) + 1


def test_oracle_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    table, ids, dy = rng.standard_normal((9, 5)), rng.integers(0, 9, 40), rng.standard_normal((40, 5))
    t = torch.from_numpy(table).requires_grad_()
    out = torch.nn.functional.embedding(torch.from_numpy(ids), t) * 3.0
    out.backward(torch.from_numpy(dy))
    assert np.array_equal(eo.lookup(ids, table, 3.0), out.detach().numpy())
    g, size, count = eo.gradient(ids, dy, 9, 3.0)
    assert np.allclose(g, t.grad.numpy(), rtol=0, atol=1e-13) and count.sum() == 40 and (size >= np.abs(g) - 1e-13).all()
    assert np.array_equal(eo.lookup(np.array([-1, 4, 5, 13, 14]), table, 1.0, first=5), np.stack([0 * table[0]] * 2 + [table[0], table[8], 0 * table[0]]))
    assert eo.gradient(np.array([-1, 4, 14]), dy[:3], 9, 1.0, first=5)[2].sum() == 0


def _look(ids=A, nb=8, n=100, first=0, table=2 * A, dt=0, rows=50, cols=200, ld=200, scale=1.0, out=3 * A, odt=0, old=200):
    return mh.lib.muonh_embedding(ids, nb, n, first, table, dt, rows, cols, ld, scale, out, odt, old, None)


@pytest.mark.parametrize("kw,code", [
    (dict(nb=2), mh.MUONH_EINVAL), (dict(n=-1), mh.MUONH_ESHAPE), (dict(n=BIG), mh.MUONH_ESHAPE),
    (dict(first=-1), mh.MUONH_EINVAL), (dict(dt=2), mh.MUONH_EINVAL), (dict(odt=2), mh.MUONH_EINVAL),
    (dict(rows=-1), mh.MUONH_ESHAPE), (dict(rows=BIG), mh.MUONH_ESHAPE), (dict(rows=0), mh.MUONH_ESHAPE),
    (dict(cols=BIG, ld=BIG, old=BIG), mh.MUONH_ESHAPE), (dict(scale=float("nan")), mh.MUONH_EINVAL),
    (dict(scale=float("inf")), mh.MUONH_EINVAL), (dict(ids=None), mh.MUONH_EINVAL), (dict(ids=A + 4), mh.MUONH_EINVAL),
    (dict(nb=4, ids=A + 2), mh.MUONH_EINVAL), (dict(table=None), mh.MUONH_EINVAL), (dict(out=None), mh.MUONH_EINVAL),
    (dict(table=2 * A + 2), mh.MUONH_EINVAL), (dict(ld=199), mh.MUONH_EINVAL), (dict(old=199), mh.MUONH_EINVAL),
    (dict(old=(1 << 36) + 1), mh.MUONH_EINVAL), (dict(out=2 * A + 49 * 800), mh.MUONH_EALIAS), (dict(out=A + 400), mh.MUONH_EALIAS),
])
def test_lookup_refuses(kw, code):
    assert _look(**kw) == code
    assert mh.lib.muonh_last_error()


def test_lookup_of_nothing_is_a_no_op():
    assert _look(n=0, ids=None, table=None, out=None) == mh.MUONH_OK
    assert _look(cols=0, ld=0, old=0, ids=None, table=None, out=None) == mh.MUONH_OK


def _back(ids=A, nb=8, n=2000, first=0, dy=2 * A, dt=0, dld=200, scale=1.0, g=3 * A, rows=50, cols=200, ld=200, acc=1, ws=4 * A,
          size=1 << 34):
    return mh.lib.muonh_embedding_backward(ids, nb, n, first, dy, dt, dld, scale, g, rows, cols, ld, acc, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(nb=16), mh.MUONH_EINVAL), (dict(n=-1), mh.MUONH_ESHAPE), (dict(n=BIG), mh.MUONH_ESHAPE),
    (dict(first=-5), mh.MUONH_EINVAL), (dict(dt=256), mh.MUONH_EINVAL), (dict(rows=BIG), mh.MUONH_ESHAPE),
    (dict(cols=-1), mh.MUONH_ESHAPE), (dict(scale=float("-inf")), mh.MUONH_EINVAL), (dict(ids=None), mh.MUONH_EINVAL),
    (dict(dy=None), mh.MUONH_EINVAL), (dict(g=None), mh.MUONH_EINVAL), (dict(g=3 * A + 2), mh.MUONH_EINVAL),
    (dict(dy=2 * A + 1, dt=1), mh.MUONH_EINVAL), (dict(dld=199), mh.MUONH_EINVAL), (dict(ld=199), mh.MUONH_EINVAL),
    (dict(n=1 << 24, cols=1 << 15, dld=1 << 15, ld=1 << 15), mh.MUONH_ESHAPE),
    (dict(ws=None), mh.MUONH_EWORKSPACE), (dict(ws=4 * A + 64), mh.MUONH_EWORKSPACE), (dict(size=1000), mh.MUONH_EWORKSPACE),
    (dict(g=2 * A + 800), mh.MUONH_EALIAS), (dict(g=A - 800), mh.MUONH_EALIAS), (dict(ws=2 * A), mh.MUONH_EALIAS),
    (dict(ws=A), mh.MUONH_EALIAS), (dict(ws=3 * A + 256), mh.MUONH_EALIAS),
])
def test_backward_refuses(kw, code):
    assert _back(**kw) == code
    assert mh.lib.muonh_last_error()


def test_backward_of_nothing_is_a_no_op():
    assert _back(rows=0, ids=A, dy=None, g=None, ws=None) == mh.MUONH_OK
    assert _back(cols=0, ids=None, dy=None, g=None, ws=None) == mh.MUONH_OK
    assert _back(n=0, ids=None, dy=None, ws=None) == mh.MUONH_OK  # accumulate: nothing to add


def test_workspace():
    f = mh.lib.muonh_embedding_backward_workspace_bytes
    assert f(0, 5) == f(5, 0) == f(-1, 5) == f(BIG, 5) == f(1 << 24, 1 << 15) == 0
    sizes = [f(n, 2048) for n in (1, 777, 8192, 16384, 16385, 1 << 20)]
    assert sizes[0] == sizes[1] == 0 and all(0 < s < 160 << 20 for s in sizes[2:])
    assert f(1024, 2048) == 0 < f(1025, 2048)
    assert _back(n=100, ws=None, size=0, g=2 * A) == mh.MUONH_EALIAS  # no workspace asked for


def test_python_refuses():
    torch = pytest.importorskip("torch")
    ids, t = torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        mh.embedding(ids, t)
    with pytest.raises(ValueError, match="GPU"):
        mh.embedding_backward(ids, torch.zeros(3, 8), t)
    with pytest.raises(TypeError):
        mh.embedding(ids, t.double())
    with pytest.raises(TypeError):
        mh.embedding_backward(ids, torch.zeros(3, 8), t.bfloat16())


@pytest.mark.parametrize("first", [-(1 << 64), -(1 << 64) + 5, -(1 << 63) - 1, 1 << 63, 1 << 64, float("inf"), float("-inf"), float("nan"), 0.5])
def test_first_that_the_call_could_not_hold(first):
    """64 bits signed: the call would take the value modulo 2^64, -2^64 as 0."""
    torch = pytest.importorskip("torch")
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="first"):
        mh._ids(ids, ids.device, first)


@pytest.mark.parametrize("first", [0, 5, (1 << 63) - 1, -1, -(1 << 63), 3.0, np.int64(7)])
def test_first_that_it_holds(first):
    """Those below zero are refused by the call itself."""
    torch = pytest.importorskip("torch")
    ids = torch.zeros(3, dtype=torch.int32)
    assert mh._ids(ids, ids.device, first) == 4
    assert _look(first=int(first), n=0) == (mh.MUONH_OK if first >= 0 else mh.MUONH_EINVAL)
