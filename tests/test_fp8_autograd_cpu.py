"""What autograd is told of the 8-bit operators, without a GPU: nothing is
recorded, and the versions of tensors that were written into move on. The
launches are stubbed out."""
from __future__ import annotations

from types import SimpleNamespace

import pytest

import orthogonalized_updates_amd as mh

torch = pytest.importorskip("torch")


@pytest.fixture
def matrix(monkeypatch):
    """An Fp8Matrix on host memory; launches do nothing."""
    empty = torch.empty
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda s, dtype, device: empty(s, dtype=dtype))
        q = mh.Fp8Matrix.empty(4, 300, "rows")
    monkeypatch.setattr(mh, "_on_device", lambda *a: None)
    return q


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_product_moves_the_version_of_out(matrix, dtype):
    out = torch.zeros(4, 4, dtype=dtype)
    for accumulate in (False, True):
        v = out._version
        assert mh.fp8_matmul(matrix, matrix, out=out, accumulate=accumulate) is out
        assert out._version == v + 1
    # a part of a tensor moves the whole
    whole = torch.zeros(8, 4, dtype=dtype)
    mh.fp8_matmul(matrix, matrix, out=whole[2:6])
    assert whole._version == 1
    assert not mh.fp8_matmul(matrix, matrix, out_dtype=dtype).requires_grad


def test_a_saved_out_is_refused_by_the_backward_pass(matrix):
    x = torch.ones(4, 4, requires_grad=True)
    out = torch.ones(4, 4)
    y = (x * out).sum()  # saves out
    mh.fp8_matmul(matrix, matrix, out=out, accumulate=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_quantized_weights_move_the_version_of_their_set(monkeypatch):
    monkeypatch.setattr(mh, "_on_device", lambda *a: None)
    opt = object.__new__(mh.MuonH)
    opt.device, opt.plan, opt._ptr_array = "cuda:0", SimpleNamespace(handle=1), lambda name, tensors: 2
    opt.torch = SimpleNamespace(cuda=SimpleNamespace(current_stream=lambda dev: None))
    memory = torch.zeros(64, dtype=torch.uint8)
    codes = memory[:32].view(torch.float8_e4m3fn)
    memory.record_stream = lambda s: None
    opt._quantize([], SimpleNamespace(memory=memory, arrays=[1, 2, 3, 4]))
    assert codes._version == 1
