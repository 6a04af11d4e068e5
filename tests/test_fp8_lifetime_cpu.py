"""What the 8-bit weight set's memory hangs on, without a GPU: its pointer
arrays live as long as its matrices, and every call that reads them records
the stream it launches on."""
from __future__ import annotations

import ctypes
from types import SimpleNamespace

import pytest

import orthogonalized_updates_amd as mh

torch = pytest.importorskip("torch")


@pytest.fixture
def on_the_host(monkeypatch):
    """Fp8Weights on host memory: its matrices without the check for a GPU."""
    monkeypatch.setattr(mh, "Fp8Matrix", lambda codes, scales, shape, block: SimpleNamespace(
        codes=codes, scales=scales, shape=shape, block=block))


@pytest.mark.parametrize("transposed", [True, False])
def test_pointer_arrays_live_in_the_matrices_memory(on_the_host, transposed):
    shapes, order = [(5, 300), (129, 7), (5, 300)], [0, 2, 1]
    ws = mh.Fp8Weights(shapes, torch.device("cpu"), transposed, order)
    matrices = [ws.weights, ws.transposed]
    store = ws.weights[1].codes.untyped_storage()
    lo, hi = store.data_ptr(), store.data_ptr() + store.nbytes()
    assert ws.span == (lo, hi)
    used = [(m.data_ptr(), m.data_ptr() + m.numel()) for q in ws.weights + ws.transposed for m in (q.codes, q.scales)]
    assert len(ws.arrays) == 4
    for i, at in enumerate(ws.arrays):
        if i >= 2 and not transposed:
            assert at is None
            continue
        used.append((at, at + 8 * len(order)))
        held = (ctypes.c_int64 * len(order)).from_address(at)
        part = ("codes", "scales")[i % 2]
        assert list(held) == [getattr(matrices[i // 2][c], part).data_ptr() for c in order]
    used.sort()
    assert lo <= used[0][0] and used[-1][1] <= hi
    assert all(a[1] <= b[0] for a, b in zip(used, used[1:]))
    # clearing the matrices' storage leaves the pointers
    before = [list((ctypes.c_int64 * len(order)).from_address(at)) for at in ws.arrays if at]
    ws.storage.fill_(0xA5)
    assert before == [list((ctypes.c_int64 * len(order)).from_address(at)) for at in ws.arrays if at]
    # and a matrix alone keeps them
    at, keep = ws.arrays[0], ws.weights[2].scales
    del ws, matrices, store
    assert list((ctypes.c_int64 * len(order)).from_address(at)) == before[0]
    assert keep.untyped_storage().data_ptr() == lo


def test_every_quantization_records_its_stream(monkeypatch):
    log = []
    stream = object()
    opt = object.__new__(mh.MuonH)
    opt.device = "cuda:1"
    opt.torch = SimpleNamespace(cuda=SimpleNamespace(current_stream=lambda dev: (stream, dev)))
    opt.plan = SimpleNamespace(handle=11)
    opt._ptr_array = lambda name, tensors: 12
    out = SimpleNamespace(memory=SimpleNamespace(record_stream=lambda s: log.append(("record", s))), arrays=[1, 2, 3, 4])
    monkeypatch.setattr(mh, "_on_device", lambda t, dev, fn, *args: log.append(("launch", dev, args)))
    opt._quantize([], out)
    assert log == [("record", (stream, "cuda:1")), ("launch", "cuda:1", (11, 12, 1, 2, 3, 4))]
