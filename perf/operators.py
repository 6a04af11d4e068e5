"""Measured cases of the block-scaled 8-bit operators: quantization to e4m3
with a power-of-two scale per block of 128, products of such matrices (the
forward, data-gradient and weight-gradient products of a linear layer, single
tokens included), and the quantization of every weight of a MuonH plan.

Formats. A matrix of rows x cols is held as e4m3 codes, rows x ld with
ld = cols rounded up to 128 and zeros past cols, and E8M0 scales (the byte
e + 127 stands for 2^e), one per 1 x 128 group of a row ("rows") or per
128 x 128 block ("tiles"), each row of scales padded to a multiple of 4.
For a block whose largest magnitude is a, e is the smallest integer >= -126
with a <= 448 * 2^e; a code is x * 2^-e rounded once to e4m3, ties to even.
The product is C[m][n] = sum_k A[m][k] B[n][k] over dequantized values.

Tokens per pass: 2 sequences of 4,096. Layer sizes: the Qwen3-style 2B set
(2048, 512, 6144) and the 4096 x 14336 set of this repository's workloads.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
TOKENS = 8192
LAYER = ((2048, 2048), (512, 2048), (512, 2048), (2048, 2048), (6144, 2048), (6144, 2048), (2048, 6144))


def listed():
    return [
        # one decoded token's activations, on the way into a projection: latency
        dict(name="quantize token", op="quantize", rows=1, cols=2048, dtype="bf16", forms="plain"),
        # a layer's input activations in training: the forward product reads
        # them grouped along features, the weight gradient along tokens
        dict(name="quantize activations", op="quantize", rows=TOKENS, cols=2048, dtype="bf16", forms="both"),
        # an fp32 gradient of odd sizes, for the weight gradient only
        dict(name="quantize ragged", op="quantize", rows=4099, cols=1001, dtype="fp32", forms="transposed"),
        # the weights of one layer after an optimizer step, both orientations
        dict(name="weights of a layer", op="weights", sets="layer", count=1),
        # large matrices, wide and tall
        dict(name="weights of large matrices", op="weights", sets="large", count=2),
        # a decoded token through the gate projection
        dict(name="product token", op="product", m=1, n=6144, k=2048, a="rows", b="tiles", dtype="bf16", add=False),
        # forward product of the gate projection
        dict(name="product forward", op="product", m=TOKENS, n=6144, k=2048, a="rows", b="tiles", dtype="bf16", add=False),
        # its gradient with respect to the activations
        dict(name="product data gradient", op="product", m=TOKENS, n=2048, k=6144, a="rows", b="tiles", dtype="bf16", add=False),
        # its weight gradient, added to the micro-batches before it
        dict(name="product weight gradient", op="product", m=6144, n=2048, k=TOKENS, a="rows", b="rows", dtype="fp32", add=True),
        # weight gradient of the key projection: few outputs, long sums
        dict(name="product key gradient", op="product", m=512, n=2048, k=TOKENS, a="rows", b="rows", dtype="fp32", add=True),
        # a ragged batch through odd sizes
        dict(name="product ragged", op="product", m=777, n=1003, k=1501, a="rows", b="rows", dtype="fp32", add=False),
        # one linear layer's whole training pass: quantize the input and the
        # output gradient, the three products, the weight gradient added to G
        dict(name="linear training pass", op="linear", tokens=TOKENS, n=14336, k=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "weights", "product", "product", "product", "linear"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 64, 8192), dtype=rng.choice(["bf16", "fp32"]),
                    forms=rng.choice(["plain", "transposed", "both"]))
    if op == "weights":
        return dict(op=op, sets="custom", rows=_log(rng, 100, 8192), cols=_log(rng, 100, 8192), count=rng.randint(1, 5))
    if op == "product":
        return dict(op=op, m=_log(rng, 1, 12288), n=_log(rng, 64, 8192), k=_log(rng, 64, 12288),
                    a="rows", b=rng.choice(["rows", "tiles"]), dtype=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.4)
    return dict(op=op, tokens=_log(rng, 16, TOKENS), n=_log(rng, 256, 8192), k=_log(rng, 256, 8192))


def _up(v, m):
    return -(-v // m) * m


def _shapes(case):
    if case["sets"] == "layer":
        return list(LAYER) * case["count"]
    if case["sets"] == "large":
        return [(4096, 14336), (14336, 4096)] * case["count"]
    return [(case["rows"], case["cols"]), (case["cols"], case["rows"])] * case["count"]


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        out = 2 if case["forms"] == "both" else 1
        return {"bytes": n * (4 if case["dtype"] == "fp32" else 2) + out * (n + n / BLOCK), "flops": 2 * n * out}
    if case["op"] == "weights":
        n = sum(r * c for r, c in _shapes(case))
        return {"bytes": n * 6, "flops": 3 * n}
    size = lambda d: 4 if d == "fp32" else 2  # noqa: E731
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * (1 + 1 / BLOCK) + m * n * size(case["dtype"]) * (2 if case["add"] else 1), "flops": 2 * m * n * k}
    t, n, k = case["tokens"], case["n"], case["k"]
    return {"bytes": t * (n + k) * 2 + 2 * n * k + t * (n + k) * 2 + n * k * 8, "flops": 6 * t * n * k}


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed % 1000003) + 17)
    return g


def _activations(g, rows, cols):
    """Normal values with a spread of channel sizes, a few of them large."""
    chan = torch.exp(0.6 * torch.randn(cols, device="cuda", generator=g))
    return torch.randn(rows, cols, device="cuda", generator=g) * chan


def _gradients(g, rows, cols):
    """Small, with token weights that differ by orders of magnitude."""
    tok = torch.exp(1.5 * torch.randn(rows, 1, device="cuda", generator=g))
    return torch.randn(rows, cols, device="cuda", generator=g) * tok * 1e-4


def _weights(g, rows, cols):
    return torch.randn(rows, cols, device="cuda", generator=g) * 0.02


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "quantize":
        s["x"] = (_gradients if case["forms"] == "transposed" else _activations)(g, case["rows"], case["cols"]).to(DTYPES[case["dtype"]])
    elif case["op"] == "weights":
        s["w"] = [_weights(g, r, c) for r, c in _shapes(case)]
        if own:
            import orthogonalized_updates_amd as mh
            s["opt"] = mh.MuonH([tuple(w.shape) for w in s["w"]])
            s["set"] = s["opt"].fp8_weights()
    elif case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        x = _gradients(g, m, k) * 1e4 if case["add"] else _activations(g, m, k)
        w = _weights(g, n, k) if case["b"] == "tiles" else _activations(g, n, k)
        s["a"], s["b"] = _held(x, case["a"]), _held(w, case["b"])
        if case["add"]:
            s["c"] = (torch.randn(m, n, device="cuda", generator=g) * math.sqrt(k)).to(DTYPES[case["dtype"]])
    else:
        t, n, k = case["tokens"], case["n"], case["k"]
        s["x"] = _activations(g, t, k).to(torch.bfloat16)
        s["dy"] = _gradients(g, t, n).to(torch.bfloat16)
        w = _weights(g, n, k)
        s["w"], s["wt"] = _held(w, "tiles"), _held(w.t(), "tiles")
        s["g"] = torch.randn(n, k, device="cuda", generator=g) * 1e-2
    return s


def _held(x, block):
    """x as the codes and scales that a program holds, in the stored layout."""
    rows, cols = x.shape
    codes, exps = _quantize(x, block)
    c = torch.zeros(rows, _up(cols, BLOCK), device="cuda", dtype=torch.uint8)
    c[:, :cols] = codes.view(torch.uint8)
    e = torch.zeros(exps.shape[0], _up(exps.shape[1], 4), device="cuda", dtype=torch.uint8)
    e[:, :exps.shape[1]] = (exps + 127).to(torch.uint8)
    return {"codes": c.view(torch.float8_e4m3fn), "scales": e.view(torch.float8_e8m0fnu), "shape": (rows, cols), "block": block}


# ---- the plain form ---------------------------------------------------------
def _pow2(e):
    """2^e in 64 bits from its bit pattern: exact, which pow() need not be."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exponents(amax):
    """The smallest e >= -126 with amax <= 448 * 2^e = 0.875 * 2^(e + 9)."""
    m, ex = torch.frexp(amax)
    e = ex - 9 + (m > 0.875).to(ex.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp_min(-126)


def _spread(exps, rows, cols, block):
    """One value for each block, as one for each entry of a rows x cols matrix."""
    if block == "tiles":
        exps = exps.repeat_interleave(BLOCK, 0)[:rows]
    return exps.repeat_interleave(BLOCK, 1)[:, :cols]


def _quantize(x, block):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    high = _up(rows, BLOCK) if block == "tiles" else rows
    a = torch.zeros(high, nb * BLOCK, device=x.device)
    a[:rows, :cols] = x.float().abs()
    a = a.view(high, nb, BLOCK).amax(2)
    if block == "tiles":
        a = a.view(high // BLOCK, BLOCK, nb).amax(1)
    exps = _exponents(a)
    v = x.double() * _pow2(-_spread(exps, rows, cols, block))
    return v.float().to(torch.float8_e4m3fn), exps


def _values(h):
    rows, cols = h["shape"]
    exps = h["scales"].view(torch.uint8).to(torch.int32)[:, :-(-cols // BLOCK)] - 127
    return _value(h["codes"][:, :cols], exps, h["block"])


def _value(codes, exps, block):
    rows, cols = codes.shape
    return codes.float() * _spread(_pow2(exps).float(), rows, cols, block)


def _out(codes, exps):
    return {"codes": codes, "scales": (exps + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _forms(x, block, forms):
    got = {}
    if forms != "transposed":
        got["plain"] = _out(*_quantize(x, block))
    if forms != "plain":
        got["transposed"] = _out(*_quantize(x.t(), block))
    return got


def _view(q):
    return {"codes": q.codes[:, :q.shape[1]], "scales": q.scales[:, :-(-q.shape[1] // BLOCK)]}


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "quantize":
        return _forms(s["x"], "rows", case["forms"])
    if case["op"] == "weights":
        return [_forms(w, "tiles", "both") for w in s["w"]]
    if case["op"] == "product":
        c = _values(s["a"]) @ _values(s["b"]).t()
        if case["add"]:
            s["c"].copy_(s["c"].float() + c)
            return s["c"]
        return c.to(DTYPES[case["dtype"]])
    x, dy = s["x"], s["dy"]
    y = _value(*_quantize(x, "rows"), "rows") @ _values(s["w"]).t()
    dx = _value(*_quantize(dy, "rows"), "rows") @ _values(s["wt"]).t()
    s["g"].add_(_value(*_quantize(dy.t(), "rows"), "rows") @ _value(*_quantize(x.t(), "rows"), "rows").t())
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "g": s["g"]}


def _matrix(mh, h):
    return mh.Fp8Matrix(h["codes"], h["scales"], h["shape"], h["block"])


def _run_own(s, case):
    import orthogonalized_updates_amd as mh
    if case["op"] == "quantize":
        q, qt = mh.fp8_quantize(s["x"], forms=case["forms"])
        got = {} if q is None else {"plain": _view(q)}
        return got if qt is None else dict(got, transposed=_view(qt))
    if case["op"] == "weights":
        s["opt"].quantize_weights(s["w"], s["set"])
        return [{"plain": _view(q), "transposed": _view(qt)} for q, qt in zip(s["set"].weights, s["set"].transposed)]
    if case["op"] == "product":
        a, b = _matrix(mh, s["a"]), _matrix(mh, s["b"])
        if case["add"]:
            return mh.fp8_matmul(a, b, out=s["c"], accumulate=True)
        return mh.fp8_matmul(a, b, out_dtype=DTYPES[case["dtype"]])
    x, xt = mh.fp8_quantize(s["x"], forms="both")
    dy, dyt = mh.fp8_quantize(s["dy"], forms="both")
    y = mh.fp8_matmul(x, _matrix(mh, s["w"]))
    dx = mh.fp8_matmul(dy, _matrix(mh, s["wt"]))
    mh.fp8_matmul(dyt, xt, out=s["g"], accumulate=True)
    return {"y": y, "dx": dx, "g": s["g"]}


# ---- from the definition, in 64 bits ----------------------------------------
def _two(e):
    """Exact powers of two: 1 scaled by numpy's ldexp through a table."""
    table = torch.from_numpy(np.ldexp(1.0, np.arange(-160, 161))).to(e.device)
    return table[(e + 160).long()]


def _grid(v):
    """v rounded to the e4m3 grid: 3 mantissa bits from 2^-6 up, steps of 2^-9 below."""
    size = v.abs()
    top = torch.floor(torch.log2(torch.where(size > 0, size, torch.ones_like(size))))
    top = torch.where(_two(top) > size, top - 1, top)  # log2 rounded up past a power of two
    top = torch.where(_two(top + 1) <= size, top + 1, top)
    step = _two(top.clamp_min(-6.0) - 3)
    return torch.round(v / step) * step


def _exact_quantize(x, block):
    """(values on the e4m3 grid, scales, both spread and by block), all in 64 bits."""
    x = x.double()
    rows, cols = x.shape
    br = BLOCK if block == "tiles" else 1
    p = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % br))
    p = p.reshape(p.shape[0] // br, br, p.shape[1] // BLOCK, BLOCK)
    a = p.abs().amax(3, keepdim=True).amax(1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / 448.0))
    e = torch.where(a > 448.0 * _two(e), e + 1, e)
    e = torch.where(a <= 448.0 * _two(e - 1), e - 1, e)
    e = torch.where(a > 0, e, torch.full_like(e, -126.0)).clamp_min(-126.0)
    scale = _two(e)
    codes = _grid(p / scale)
    flat = lambda t: t.reshape(t.shape[0] * t.shape[1], t.shape[2] * t.shape[3])  # noqa: E731
    return flat(codes)[:rows, :cols], flat(scale), flat(codes * scale)[:rows, :cols]


def _exact_values(h):
    """Codes and scale bytes read bit by bit."""
    rows, cols = h["shape"]
    c = h["codes"].view(torch.uint8)[:, :cols].to(torch.int64)
    mant, ex = (c & 7).double(), ((c >> 3) & 15).double()
    size = torch.where(ex > 0, (8 + mant) * _two(ex - 10), mant * (2.0 ** -9))
    v = torch.where(c >= 128, -size, size)
    e = _two(h["scales"].view(torch.uint8).double() - 127)
    br = BLOCK if h["block"] == "tiles" else 1
    i = torch.arange(rows, device=c.device) // br
    j = torch.arange(cols, device=c.device) // BLOCK
    return v * e[i][:, j]


def exact(case, seed):
    s = prepare(case, seed)

    def forms(x, block, which):
        got = {}
        for name, v in (("plain", x), ("transposed", x.t())):
            if which in (name, "both"):
                codes, scale, _ = _exact_quantize(v, block)
                got[name] = {"codes": codes, "scales": scale}
        return got

    if case["op"] == "quantize":
        return forms(s["x"], "rows", case["forms"])
    if case["op"] == "weights":
        return [forms(w, "tiles", "both") for w in s["w"]]
    if case["op"] == "product":
        c = torch.matmul(_exact_values(s["a"]), _exact_values(s["b"]).t().contiguous())
        return c + s["c"].double() if case["add"] else c
    x, dy = s["x"], s["dy"]
    times = lambda a, b: torch.matmul(a, b.t().contiguous())  # noqa: E731
    q = lambda t: _exact_quantize(t, "rows")[2]  # noqa: E731
    return {"y": times(q(x), _exact_values(s["w"])), "dx": times(q(dy), _exact_values(s["wt"])),
            "g": s["g"].double() + times(q(dy.t()), q(x.t()))}
