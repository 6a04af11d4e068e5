"""Embedding lookup and its gradient on the GPU against the fp64 oracle.

Lookup: scale * entry in fp32, half a step u = 2^-24, then half a step of the
result's type. Gradient: a row of c tokens is a sum of c terms and the old value, in
some order: c + 2 roundings at most on any term, the scale and the last sum among them:
(c + 2) u * (sum of magnitudes). Sums of small whole numbers are exact in any
order: with those, results are equal bit for bit.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import embedding_oracle as eo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def mh():
    import orthogonalized_updates_amd
    return orthogonalized_updates_amd


def f64(t):
    return t.double().cpu().numpy()


def normal(rows, cols, seed, dtype="fp32"):
    x = np.random.default_rng((seed, rows, cols)).standard_normal((rows, cols))
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()


def whole(rows, cols, seed, dtype="fp32"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-8, 9, (rows, cols), device="cuda", generator=g).to(DT[dtype])


def ids_of(kind, n, rows, seed, dtype=torch.int64):
    rng = np.random.default_rng((seed, n, rows))
    if kind == "same":
        v = np.full(n, rows // 2)
    elif kind == "distinct":
        v = rng.permutation(max(n, rows))[:n] % rows
    elif kind == "frequent":
        v = np.minimum((np.exp(rng.random(n) * np.log(rows))).astype(np.int64), rows) - 1
    elif kind == "runs":  # of lengths around the chunks' and multiples of them
        v = np.repeat(rng.integers(0, rows, n), rng.integers(1, 40, n))[:n]
    elif kind == "none":
        v = rng.choice([-1, rows, rows + 5, -(1 << 31), (1 << 31) - 1], n)
    else:  # mixed
        v = np.where(rng.random(n) < 0.3, rng.choice([-1, rows, -(1 << 31), (1 << 31) - 1], n), rng.integers(0, min(rows, 5), n))
    return torch.from_numpy(v.astype(np.int64)).to(dtype).cuda()


KINDS = ["same", "distinct", "frequent", "runs", "none", "mixed"]


@pytest.mark.parametrize("table,out", [("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (1, 500, 2048), (5, 7, 3), (100, 33, 64), (777, 5003, 1001), (33, 300, 8200), (1500, 40, 129)])
def test_lookup(n, rows, cols, table, out):
    t = normal(rows, cols, 1, table)
    for kind in ("frequent", "mixed"):
        for dtype in (torch.int64, torch.int32):
            ids = ids_of(kind, n, rows, 2, dtype)
            y = mh().embedding(ids, t, scale=3.25, out_dtype=DT[out])
            want = eo.lookup(ids.cpu().numpy(), f64(t), 3.25)
            assert y.shape == (n, cols) and y.dtype == DT[out]
            assert (np.abs(f64(y) - want) <= (U + HALF[y.dtype]) * np.abs(want)).all()
    assert torch.equal(mh().embedding(ids_of("distinct", n, rows, 3), t), t[ids_of("distinct", n, rows, 3)])


def test_lookup_shapes_strides_and_parts_of_a_table():
    t = normal(50, 300, 1)
    ids = ids_of("frequent", 24, 50, 4).view(2, 3, 4)
    want = mh().embedding(ids, t, scale=2.0)
    assert want.shape == (2, 3, 4, 300) and torch.equal(want, 2 * t[ids])
    wide = torch.full((24, 311), 7.0, device="cuda")
    base = normal(50, 307, 5)
    base[:, 3:303] = t
    got = mh().embedding(ids.view(24), base[:, 3:303], scale=2.0, out=wide[:, 5:305])
    assert torch.equal(got, want.view(24, 300)) and (wide[:, :5] == 7).all() and (wide[:, 305:] == 7).all()
    # a table split by rows: each id is found in one part, the others give zeros
    parts = [mh().embedding(ids, t[a:b], scale=2.0, first=a) for a, b in ((0, 17), (17, 18), (18, 50))]
    assert torch.equal(parts[0] + parts[1] + parts[2], want)
    assert (mh().embedding(ids, t, first=1 << 62) == 0).all()
    huge = torch.tensor([-(1 << 63), (1 << 63) - 1, -1, 49], device="cuda")
    assert torch.equal(mh().embedding(huge, t), torch.stack([torch.zeros(300, device="cuda")] * 3 + [t[49]]))


def test_values_pass_through():
    t = torch.tensor([[float("nan"), float("inf"), -float("inf"), -0.0, 1e-45, 3.4e38]], device="cuda")
    assert torch.equal(mh().embedding(torch.tensor([0, 5], device="cuda"), t).view(torch.int32), torch.stack([t[0], torch.zeros(6, device="cuda")]).view(torch.int32))


# up to 1024 tokens in one launch; else chunks of 4 to 64 tokens, in the order of one launch up to 32768 tokens (4, 8, 16 or 32 a
# thread), then of passes of 8 bits
SIZES = [(1, 1, 1), (1, 300, 2048), (2, 3, 5), (4, 4, 64), (5, 7, 128), (9, 2, 129), (13, 300, 520), (100, 257, 1001), (777, 5003, 1001),
         (1000, 256, 2048), (1024, 300, 520), (1025, 300, 520), (1024, 40000, 6), (4099, 1000, 100), (3000, 90, 4096), (16384, 3000, 64), (16385, 3000, 64), (20000, 255, 40), (20000, 256, 40),
         (20000, 257, 40), (50001, 70000, 24), (140000, 66000, 136), (70000, 1 << 24, 1), (9000, 151936, 8),
         (4096, 700, 16), (4097, 700, 16), (8192, 90000, 9), (8193, 500, 24), (32768, 40000, 8), (32769, 40000, 8)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_gradient_of_whole_numbers_is_exact(n, rows, cols, kind):
    """Against index_add_ in 64 bits; sums stay below 2^24."""
    ids = ids_of(kind, n, rows, 1, torch.int32 if n % 2 else torch.int64)
    dy = whole(n, cols, 2, "bf16" if cols % 2 == 0 else "fp32")
    old = whole(rows, cols, 3)
    keep = (ids >= 0) & (ids < rows)
    want = torch.zeros(rows, cols, dtype=torch.float64, device="cuda").index_add_(0, ids[keep].long(), dy[keep].double() * 0.5)
    got = torch.full((rows, cols), float("nan"), device="cuda")
    assert mh().embedding_backward(ids, dy, got, scale=0.5) is got
    assert torch.equal(got.double(), want)
    got = mh().embedding_backward(ids, dy, old.clone(), scale=0.5, accumulate=True)
    assert torch.equal(got.double(), want + old.double())


# several slabs of columns, where 4 waves join a row's sums, up to the most workgroups that do; one slab with as many
MORE_SIZES = [(8192, 3000, 2048), (30000, 400, 601), (4000, 150000, 2047), (33000, 500, 520), (70000, 300, 1030), (16000, 900, 500),
              (32768, 700, 300), (40000, 900, 130), (140000, 60, 20)]


@pytest.mark.parametrize("kind", ["same", "frequent", "runs", "mixed"])
@pytest.mark.parametrize("n,rows,cols", MORE_SIZES)
def test_gradient_of_many_chunks_is_exact(n, rows, cols, kind):
    test_gradient_of_whole_numbers_is_exact(n, rows, cols, kind)


@pytest.mark.parametrize("kind", ["distinct", "frequent", "many frequent", "one of them"])
@pytest.mark.parametrize("n", [1025, 4096, 5000, 16384, 32768])
def test_gradient_of_rows_that_share_a_bucket(n, kind):
    """The worst ids for the order of the tokens: products with its multiplier that differ in their low 16 bits only."""
    rows, rng = 1 << 24, np.random.default_rng((n, 9))
    inverse = pow(0x9E3779, -1, 1 << 24)
    here = (77 << 16 | rng.permutation(1 << 16)) * inverse % rows
    v = here[:n].copy()
    if kind == "frequent":  # one row's for the most part
        v = np.where(rng.random(n) < 0.9, here[0], v)
    elif kind == "many frequent":
        v = np.where(rng.random(n) < 0.8, here[rng.integers(0, 9, n)], v)
    elif kind == "one of them":  # and other buckets' in between, few of this one's rows
        v = np.where(rng.random(n) < 0.5, here[rng.integers(0, 40, n)], rng.integers(0, rows, n))
    ids, dy = torch.from_numpy(v.astype(np.int64)).cuda(), whole(n, 2, 2)
    want = torch.zeros(rows, 2, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
    got = mh().embedding_backward(ids, dy, torch.full((rows, 2), float("nan"), device="cuda"))
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,rows,cols,kind", [(1, 5, 7, "same"), (300, 100, 129, "frequent"), (777, 503, 101, "mixed"), (2000, 7, 600, "runs"),
                                              (5000, 3, 64, "same"), (17000, 50, 33, "frequent")])
def test_gradient(n, rows, cols, kind, dtype):
    ids, dy, old = ids_of(kind, n, rows, 5), normal(n, cols, 6, dtype), normal(rows, cols, 7)
    for add in (False, True):
        got = mh().embedding_backward(ids, dy, old.clone(), scale=1.7, accumulate=add)
        want, size, count = eo.gradient(ids.cpu().numpy(), f64(dy), rows, float(np.float32(1.7)), f64(old) if add else None)
        assert (np.abs(f64(got) - want) <= (count[:, None] + 2) * U * size).all()
        again = mh().embedding_backward(ids, dy, old.clone(), scale=1.7, accumulate=add)
        assert torch.equal(got, again)
    # the derivative of the lookup: <dy, lookup(T)> is linear in T, so a difference has rounding only
    if n <= 777:
        t, d = normal(rows, cols, 8), normal(rows, cols, 9)
        f = lambda t: (dy.double() * mh().embedding(ids, t, scale=1.7, out_dtype=torch.float32).double()).sum()  # noqa: E731
        g = mh().embedding_backward(ids, dy, torch.empty_like(t), scale=1.7)
        size = float((g.abs().double() * (t.abs() + d.abs()).double()).sum()) + float((dy.abs().double().sum() * 1.7 * 10))
        assert abs(float(f(t + d) - f(t)) - float((g.double() * d.double()).sum())) <= (n + 8) * U * size


def test_strides_and_untouched_rows():
    ids = torch.tensor([[4, 9, 4], [0, 4, -1]], device="cuda")
    base = whole(6, 213, 1, "bf16")
    dy = base[:, 3:203]
    wide = torch.full((12, 205), 7.0, device="cuda")
    out = wide[:, 2:202]
    assert mh().embedding_backward(ids.view(6), dy, out, accumulate=True) is out
    want = torch.full((12, 200), 7.0, device="cuda").index_add_(0, ids.view(6)[:5], dy[:5].float())
    assert torch.equal(out, want) and (wide[:, :2] == 7).all() and (wide[:, 202:] == 7).all()
    mh().embedding_backward(ids.view(6), dy, out)
    assert torch.equal(out, want - 7) and (wide[:, :2] == 7).all() and (wide[:, 202:] == 7).all()
    three = dy.contiguous().view(2, 3, 200)
    assert torch.equal(mh().embedding_backward(ids, three, torch.empty(12, 200, device="cuda")), want - 7)
    part = mh().embedding_backward(ids, three, torch.empty(5, 200, device="cuda"), first=4)
    assert torch.equal(part, (want - 7)[4:9])


def test_nan_stays_in_its_row():
    ids = torch.tensor([1, 2, 1, 3], device="cuda")
    dy = torch.ones(4, 50, device="cuda")
    dy[1, 7] = float("nan")
    g = mh().embedding_backward(ids, dy, torch.zeros(5, 50, device="cuda"), accumulate=True)
    assert g[2, 7].isnan() and int(g.isnan().sum()) == 1 and (g[1] == 2).all()
    # a padded token's values are not read into anything
    dy[:] = float("nan")
    assert (mh().embedding_backward(torch.full((4,), -1, device="cuda"), dy, torch.empty(5, 50, device="cuda")) == 0).all()


def test_nothing():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    t = normal(5, 30, 1)
    assert mh().embedding(none, t).shape == (0, 30)
    assert torch.equal(mh().embedding_backward(none, torch.empty(0, 30, device="cuda"), t.clone(), accumulate=True), t)
    assert (mh().embedding_backward(none, torch.empty(0, 30, device="cuda"), t.clone()) == 0).all()
    assert mh().embedding(torch.zeros(2, dtype=torch.int64, device="cuda"), torch.empty(5, 0, device="cuda")).shape == (2, 0)
    assert mh().embedding_backward(torch.zeros(2, dtype=torch.int64, device="cuda"), torch.empty(2, 30, device="cuda"),
                                   torch.empty(0, 30, device="cuda")).shape == (0, 30)


def test_offsets_past_32_bits():
    rows, ld = 5, (1 << 29) + 8
    base = torch.zeros((rows - 1) * ld + 40, device="cuda")
    table = base.as_strided((rows, 40), (ld, 1))
    table.copy_(whole(rows, 40, 1))
    ids = torch.tensor([4, 0, 4, 3], device="cuda")
    dense = table.contiguous()
    assert torch.equal(mh().embedding(ids, table), dense[ids])
    dy = whole(4, 40, 2)
    mh().embedding_backward(ids, dy, table, accumulate=True)
    assert torch.equal(table.contiguous(), dense.index_add(0, ids, dy))


def test_python_refuses():
    m = mh()
    ids, t, dy = torch.zeros(3, dtype=torch.int64, device="cuda"), normal(4, 8, 1), normal(3, 8, 2)
    for call in (lambda: m.embedding(ids.cpu(), t), lambda: m.embedding(ids, t.t()), lambda: m.embedding(ids, t, out=torch.empty(3, 7, device="cuda")),
                 lambda: m.embedding(torch.zeros(6, dtype=torch.int64, device="cuda")[::2], t), lambda: m.embedding_backward(ids, dy[:2], t),
                 lambda: m.embedding(ids, t, first=1 << 64), lambda: m.embedding(ids, t, first=0.5), lambda: m.embedding_backward(ids, dy, t.clone(), first=1 << 63),
                 lambda: m.embedding(ids.view(3, 1), t, out=torch.empty(1, 3, 8, device="cuda").transpose(0, 1)[:, :, :7])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: m.embedding(ids.float(), t), lambda: m.embedding(ids, t, out_dtype=torch.half), lambda: m.embedding_backward(ids, dy.double(), t),
                 lambda: m.embedding(ids, t, out=dy, out_dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: m.embedding(ids, t, first=-1), lambda: m.embedding(ids, t, scale=float("nan")), lambda: m.embedding(ids, t, out=t[:3]),
                 lambda: m.embedding(ids, torch.empty(0, 8, device="cuda"))):
        with pytest.raises(m.MuonHError):
            call()


@pytest.mark.parametrize("n", [4, 1000, 1500, 30000, 33000])
@pytest.mark.parametrize("back", [1, 3, 5, 6, 4000])
def test_ids_at_both_ends_of_64_bits(n, back):
    """The lowest ids minus a `first` near 2^63 pass 2^64: they are below `first` all the same."""
    first, rows, cols = (1 << 63) - back, 5, 40
    rng = np.random.default_rng((n, back))
    v = np.where(rng.random(n) < 0.5, rng.integers(-(1 << 63), -(1 << 63) + 8, n), (1 << 63) - 1 - rng.integers(0, 8, n))
    row = torch.from_numpy(np.where(v >= first, v - np.where(v >= first, first, 0), rows)).cuda()
    row = torch.where(row < rows, row, rows)
    ids, t, dy = torch.from_numpy(v).cuda(), whole(rows, cols, 1), whole(n, cols, 2)
    assert torch.equal(mh().embedding(ids, t, first=first), torch.cat([t, torch.zeros(1, cols, device="cuda")])[row])
    want = torch.zeros(rows + 1, cols, device="cuda").index_add_(0, row, dy)[:rows]
    got = mh().embedding_backward(ids, dy, torch.full((rows, cols), float("nan"), device="cuda"), first=first)
    assert torch.equal(got, want)
    assert torch.equal(mh().embedding_backward(ids, dy, t.clone(), first=first, accumulate=True), t + want)


@pytest.mark.parametrize("n", [700, 17000, 33000])
def test_captured_graph_and_other_stream(n):
    ids, dy = ids_of("frequent", n, 900, 1), normal(n, 520, 2, "bf16")
    table, g = normal(900, 520, 3), torch.zeros(900, 520, device="cuda")

    def run(g):
        y = mh().embedding(ids, table, scale=2.0, out_dtype=torch.bfloat16)
        mh().embedding_backward(ids, dy, g, scale=2.0)
        mh().embedding_backward(ids, y, g, accumulate=True)
        return y

    run(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(g)
    side = torch.cuda.Stream()
    for i in range(3):
        ids.copy_(ids_of(("mixed", "runs", "same")[i], n, 900, i))
        dy.copy_(normal(n, 520, 30 + i, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = (held.clone(), g.clone())
        other = torch.empty_like(g)
        y = run(other)
        assert torch.equal(got[0], y) and torch.equal(got[1], other)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            third = torch.empty_like(g)
            run(third)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(third, other)
