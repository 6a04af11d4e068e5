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


def test_a_copied_or_moved_set_is_refused(on_the_host):
    import copy
    ws = mh.Fp8Weights([(5, 300)], torch.device("cpu"), True, [0])
    opt = object.__new__(mh.MuonH)
    opt.shapes, opt.device, opt.plan_order = [(5, 300)], torch.device("cpu"), [0]
    opt._check_fp8(ws)
    opt._check_fp8(copy.copy(ws))  # the same memory
    with pytest.raises(ValueError, match="moved"):
        opt._check_fp8(copy.deepcopy(ws))
    ws.memory.set_(ws.memory.clone())
    with pytest.raises(ValueError, match="moved"):
        opt._check_fp8(ws)


def test_every_quantization_records_its_stream(monkeypatch):
    log = []
    stream = object()
    opt = object.__new__(mh.MuonH)
    opt.device = "cuda:1"
    opt.torch = SimpleNamespace(cuda=SimpleNamespace(current_stream=lambda dev: (stream, dev)))
    opt.plan = SimpleNamespace(handle=11)
    opt._ptr_array = lambda name, tensors: 12
    out = SimpleNamespace(memory=torch.zeros(8, dtype=torch.uint8), arrays=[1, 2, 3, 4])
    out.memory.record_stream = lambda s: log.append(("record", s))
    monkeypatch.setattr(mh, "_on_device", lambda t, dev, fn, *args: log.append(("launch", dev, args)))
    opt._quantize([], out)
    assert log == [("record", (stream, "cuda:1")), ("launch", "cuda:1", (11, 12, 1, 2, 3, 4))]


@pytest.fixture
def matrix(monkeypatch):
    """An Fp8Matrix on host memory."""
    empty = torch.empty
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda s, dtype, device: empty(s, dtype=dtype))
        q = mh.Fp8Matrix.empty(4, 300, "rows")
    return q


def test_a_matrix_and_its_addresses_do_not_part(matrix):
    q = matrix
    for name in q.__slots__:
        with pytest.raises(AttributeError, match="read-only"):
            setattr(q, name, getattr(q, name))
        with pytest.raises(AttributeError, match="read-only"):
            delattr(q, name)
    assert q.shape == (4, 300) and q.desc.codes == q.codes.data_ptr() and q.desc.scales == q.scales.data_ptr()
    assert mh._held("q", q) is q.desc


@pytest.mark.parametrize("part", ["codes", "scales"])
@pytest.mark.parametrize("how", ["set", "storage", "resize"])
def test_a_matrix_whose_tensors_moved_is_refused(matrix, part, how):
    q, t = matrix, getattr(matrix, part)
    if how == "set":
        t.set_(t.clone())
    elif how == "storage":
        t.untyped_storage().resize_(0)
    else:
        t.resize_(1 << 16, 64)
    with pytest.raises(ValueError, match="a's codes or scales were moved"):
        mh.fp8_matmul(q, q)
    with pytest.raises(ValueError, match="out's codes or scales were moved"):
        mh._form("out", q, True, 4, 300, "rows", q.device)


def test_copies_have_addresses_of_their_own(matrix, monkeypatch):
    import copy
    q = matrix
    q.codes.view(torch.uint8).fill_(5)
    q.scales.view(torch.uint8).fill_(127)
    # the constructor takes GPU tensors only; the rest of it is what is tested
    monkeypatch.setattr(mh.Fp8Matrix, "__init__", lambda self, *a: self._set(*a))
    same, own = copy.copy(q), copy.deepcopy(q)
    assert same.codes is q.codes and same.desc.codes == q.desc.codes
    assert own.codes.data_ptr() != q.codes.data_ptr() and own.desc.codes == own.codes.data_ptr()
    assert own.desc.scales == own.scales.data_ptr() and own.shape == q.shape and own.block == q.block
    assert torch.equal(own.codes.view(torch.uint8), q.codes.view(torch.uint8))
