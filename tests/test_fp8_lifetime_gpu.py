"""8-bit weight sets on another stream than their own, on the GPU."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def raw(q):
    return [q.codes.view(torch.uint8).clone(), q.scales.view(torch.uint8).clone()]


def test_a_dropped_sets_matrices_are_written_on_another_stream():
    """The set is made on the default stream and written on another one behind
    other work; only its matrices are kept, and new tensors of every small
    size are made and filled on the default stream meanwhile."""
    import orthogonalized_updates_amd as mh
    shapes = [(300, 200), (64, 640), (129, 129)]
    g = torch.Generator("cuda").manual_seed(3)
    W = [torch.randn(s, device="cuda", generator=g) for s in shapes]
    opt = mh.MuonH(shapes)
    ref = opt.quantize_weights(W, opt.fp8_weights())
    want = [t for q in ref.weights + ref.transposed for t in raw(q)]
    work = torch.randn(1 << 26, device="cuda", generator=g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = opt.fp8_weights()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            work.mul_(1.0001)
        opt.quantize_weights(W, ws)
    kept = ws.weights + ws.transposed
    del ws
    filler = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in range(8, 4096, 8)]
    torch.cuda.synchronize()
    assert len(filler) and all(torch.equal(a, b) for a, b in zip([t for q in kept for t in raw(q)], want))
