"""Measured cases of the operators around the linear layers: RMS norm with the
residual's addition and an output in block-scaled 8 bits, and its gradient;
embedding lookup with scaling, and its gradient by sorted tokens;
microscaled 4-bit matrices, quantization and products.

Definitions.
  RMS norm: h = x + residual, rounded once to the residual's type (h = x without
  one); r = 1 / sqrt(mean(h^2) + eps); y = h r w. Its gradient: g = dy w,
  dh = r (g - h r mean(g h r)) + dresidual, dw = sum over rows of dy h r.
  8-bit outputs hold y as e4m3 with a scale 2^e per 128 entries of a row ("plain") or
  of a column ("transposed"): the smallest e >= -126 with max|y| <= 448 * 2^e.
  Embedding: out[t] = scale * table[ids[t]], zeros for an id that is no row;
  its gradient: G[v] (+)= scale * sum of dy[t] over the t with ids[t] = v.
  4-bit matrices: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) with a scale 2^e
  per 32 entries of a row, the smallest e >= -126 with max|x| <= 6 * 2^e; a code is
  x * 2^-e rounded once, ties to even. Stored two codes to a byte, the first in
  the low half, rows of a multiple of 256 codes; scales as bytes e + 127, a
  multiple of 8 per row; zeros past the end.
  The product is C[m][n] = sum_k A[m][k] B[n][k].

Tokens per pass: 2 sequences of 4,096. Sizes: the Qwen3-style 2B set (2048, 6144,
heads of 128, a table of 151,936 x 2048) and the 4096 x 14336 set of this repository's
workloads.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
TOKENS = 8192
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token's way into a layer: latency
        dict(name="norm token", op="norm", rows=1, cols=2048, dtype="bf16", residual=True, forms="plain"),
        # a layer's input in training: the new residual stream, and the operand
        # of the forward products and of the weight gradients
        dict(name="norm with residual in 8 bits", op="norm", rows=TOKENS, cols=2048, dtype="bf16", residual=True, forms="both"),
        # the norm of 16 heads of 128 for each token
        dict(name="norm of heads", op="norm", rows=16 * TOKENS, cols=128, dtype="bf16", residual=False, forms="none"),
        # its way back, joined with the residual's gradient
        dict(name="norm gradient", op="norm gradient", rows=TOKENS, cols=2048, dtype="bf16", residual=True),
        # a batch's tokens out of the trained table
        dict(name="embedding", op="embedding", tokens=TOKENS, vocab=151936, cols=2048, table="fp32", dtype="bf16", pad=False),
        # their gradient, added to the table's, which holds the output layer's
        dict(name="embedding gradient", op="embedding gradient", tokens=TOKENS, vocab=151936, cols=2048, dtype="bf16", add=True, pad=False),
        # odd sizes, padding among the ids, into a gradient that starts at zero
        dict(name="embedding gradient ragged", op="embedding gradient", tokens=777, vocab=5003, cols=1001, dtype="fp32", add=False, pad=True),
        # activations to 4 bits along features and along tokens, and the values that these hold
        dict(name="4 bits activations", op="values", rows=TOKENS, cols=2048, dtype="bf16", forms="both"),
        # a decoded token through a projection held in 4 bits
        dict(name="4 bits token", op="linear", m=1, n=6144, k=2048),
        # the gate projection of a batch
        dict(name="4 bits forward", op="product", m=TOKENS, n=6144, k=2048, dtype="bf16", add=False),
        # a ragged batch through odd sizes, added to what is there
        dict(name="4 bits ragged", op="product", m=777, n=1003, k=1501, dtype="fp32", add=True),
        # one linear layer's whole training pass: quantize the input and the
        # output gradient, the three products, the weight gradient added to G
        dict(name="4 bits training pass", op="training", tokens=TOKENS, n=14336, k=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm gradient", "embedding", "embedding gradient", "values", "linear", "product", "product", "training"])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 64, 8192), dtype=dtype, residual=rng.random() < 0.6,
                    forms=rng.choice(["none", "plain", "transposed", "both"]))
    if op == "norm gradient":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 64, 8192), dtype=dtype, residual=rng.random() < 0.6)
    if op == "embedding":
        return dict(op=op, tokens=_log(rng, 1, 16384), vocab=_log(rng, 100, 151936), cols=_log(rng, 64, 4096),
                    table=rng.choice(["bf16", "fp32"]), dtype=dtype, pad=rng.random() < 0.3)
    if op == "embedding gradient":
        return dict(op=op, tokens=_log(rng, 1, 16384), vocab=_log(rng, 100, 151936), cols=_log(rng, 64, 4096), dtype=dtype,
                    add=rng.random() < 0.6, pad=rng.random() < 0.3)
    if op == "values":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 64, 8192), dtype=dtype, forms=rng.choice(["plain", "transposed", "both"]))
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 256), n=_log(rng, 64, 8192), k=_log(rng, 64, 8192))
    if op == "product":
        return dict(op=op, m=_log(rng, 1, 12288), n=_log(rng, 64, 8192), k=_log(rng, 64, 12288), dtype=dtype, add=rng.random() < 0.4)
    return dict(op=op, tokens=_log(rng, 16, TOKENS), n=_log(rng, 256, 8192), k=_log(rng, 256, 8192))


def _size(dtype):
    return 4 if dtype == "fp32" else 2


def work(case):
    op = case["op"]
    if op in ("norm", "norm gradient"):
        n, e = case["rows"] * case["cols"], _size(case["dtype"])
        if op == "norm gradient":  # dy, h and the residual's gradient in, dh out
            return {"bytes": n * e * (4 if case["residual"] else 3) + case["cols"] * 8 + case["rows"] * 4, "flops": 10 * n}
        out = {"none": e, "plain": 1, "transposed": 1, "both": 2}[case["forms"]]
        return {"bytes": n * (e * (3 if case["residual"] else 1) + out) + case["cols"] * 4 + case["rows"] * 4, "flops": 5 * n}
    if op == "embedding":
        rows = min(case["tokens"], case["vocab"])
        return {"bytes": rows * case["cols"] * _size(case["table"]) + case["tokens"] * (case["cols"] * _size(case["dtype"]) + 8), "flops": case["tokens"] * case["cols"]}
    if op == "embedding gradient":
        t, d = case["tokens"], case["cols"]
        # about a third of a batch's tokens are others than those before them
        into = 2 * min(t / 3, case["vocab"]) if case["add"] else case["vocab"]
        return {"bytes": t * (d * _size(case["dtype"]) + 8) + into * d * 4, "flops": 2 * t * d}
    if op == "values":
        n, out = case["rows"] * case["cols"], 2 if case["forms"] == "both" else 1
        return {"bytes": n * (_size(case["dtype"]) + out * (2 * (0.5 + 1 / 32) + 2)), "flops": 3 * n * out}
    if op in ("linear", "product"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "linear":
            return {"bytes": m * k * 2 + n * k * (0.5 + 1 / 32) + m * n * 2, "flops": 2 * m * n * k}
        return {"bytes": (m + n) * k * (0.5 + 1 / 32) + m * n * _size(case["dtype"]) * (2 if case["add"] else 1), "flops": 2 * m * n * k}
    t, n, k = case["tokens"], case["n"], case["k"]
    return {"bytes": t * (n + k) * 2 + 2 * n * k * (0.5 + 1 / 32) + t * (n + k) * 2 + n * k * 8, "flops": 6 * t * n * k}


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed % 1000003) + 29)
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


def _ids(g, case):
    """Token ids as text has them: the i-th most frequent with a share of about
    1/i, so that the first takes some percent of a batch; -1 where padded."""
    u = torch.rand(case["tokens"], device="cuda", generator=g, dtype=torch.float64)
    ids = torch.exp(u * math.log(case["vocab"])).long().clamp_(1, case["vocab"]) - 1
    if case["pad"]:
        ids = torch.where(torch.rand(case["tokens"], device="cuda", generator=g) < 0.2, torch.full_like(ids, -1), ids)
    return ids


def prepare(case, seed):
    g = _gen(seed)
    s, op = {"case": case}, case["op"]
    if op in ("norm", "norm gradient"):
        rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["w"] = 1 + 0.2 * torch.randn(cols, device="cuda", generator=g)
        s["x"] = _activations(g, rows, cols).to(dtype)
        if op == "norm":
            s["res"] = (2 * _activations(g, rows, cols)).to(dtype) if case["residual"] else None
        else:
            s["dy"] = _gradients(g, rows, cols).to(dtype)
            s["dres"] = _gradients(g, rows, cols).to(dtype) if case["residual"] else None
            # the forward pass left the inverse root mean squares
            s["r"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
    elif op == "embedding":
        s["ids"] = _ids(g, case)
        s["table"] = _weights(g, case["vocab"], case["cols"]).to(DTYPES[case["table"]])
    elif op == "embedding gradient":
        s["ids"] = _ids(g, case)
        s["dy"] = _gradients(g, case["tokens"], case["cols"]).to(DTYPES[case["dtype"]])
        s["g"] = torch.randn(case["vocab"], case["cols"], device="cuda", generator=g) * 1e-4
    elif op == "values":
        s["x"] = (_gradients if case["forms"] == "transposed" else _activations)(g, case["rows"], case["cols"]).to(DTYPES[case["dtype"]])
    elif op == "linear":
        s["x"] = _activations(g, case["m"], case["k"]).to(torch.bfloat16)
        s["w"] = _held(_weights(g, case["n"], case["k"]))
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["b"] = _held(_activations(g, m, k)), _held(_weights(g, n, k))
        if case["add"]:
            s["c"] = (torch.randn(m, n, device="cuda", generator=g) * math.sqrt(k) * 0.02).to(DTYPES[case["dtype"]])
    else:
        t, n, k = case["tokens"], case["n"], case["k"]
        s["x"] = _activations(g, t, k).to(torch.bfloat16)
        s["dy"] = _gradients(g, t, n).to(torch.bfloat16)
        w = _weights(g, n, k)
        s["w"], s["wt"] = _held(w), _held(w.t())
        s["g"] = torch.randn(n, k, device="cuda", generator=g) * 1e-2
    return s


def _up(v, m):
    return -(-v // m) * m


def _held(x):
    """x as the codes and scales that a program holds, in the stored layout."""
    rows, cols = x.shape
    codes, exps = _quantize4(x)
    c = torch.zeros(rows, _up(cols, 256), device="cuda", dtype=torch.uint8)
    c[:, :cols] = codes
    e = torch.zeros(rows, _up(cols, 256) // 32, device="cuda", dtype=torch.uint8)
    e[:, :exps.shape[1]] = (exps + 127).to(torch.uint8)
    c = (c[:, 0::2] | c[:, 1::2] << 4).contiguous()
    return {"codes": c.view(torch.float4_e2m1fn_x2), "scales": e.view(torch.float8_e8m0fnu), "shape": (rows, cols)}


# ---- the plain form ---------------------------------------------------------
def _pow2(e):
    """2^e in 64 bits from its bit pattern: exact, which pow() need not be."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exponents(x, block, top, shift):
    """For each `block` entries of a row, the smallest e >= -126 with a <= top * 2^(e + shift), 0.5 <= top < 1."""
    rows, cols = x.shape
    nb = -(-cols // block)
    a = torch.zeros(rows, nb * block, device=x.device)
    a[:, :cols] = x.float().abs()
    a = a.view(rows, nb, block).amax(2)
    m, ex = torch.frexp(a)
    e = ex - shift + (m > top).to(ex.dtype)
    return torch.where(a > 0, e, torch.full_like(e, -126)).clamp_min(-126)


def _over_scales(x, exps, block):
    return (x.double() * _pow2(-exps.repeat_interleave(block, 1)[:, :x.shape[1]])).float()


def _quantize8(x):
    exps = _exponents(x, 128, 0.875, 9)
    return {"codes": _over_scales(x, exps, 128).to(torch.float8_e4m3fn), "scales": (exps + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _quantize4(x):
    exps = _exponents(x, 32, 0.75, 3)
    v = _over_scales(x, exps, 32)
    m = v.abs()
    over = (m > 0.25, m >= 0.75, m > 1.25, m >= 1.75, m > 2.5, m >= 3.5, m > 5)  # a value halfway takes the even code
    code = torch.stack(over).sum(0, dtype=torch.uint8)
    return code + 8 * (v < 0).to(torch.uint8), exps


def _values4(codes, exps):
    """What codes (one to a byte) and exponents stand for."""
    size = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    return size[codes.long()] * _pow2(exps).float().repeat_interleave(32, 1)[:, :codes.shape[1]]


def _values(h):
    rows, cols = h["shape"]
    c = h["codes"].view(torch.uint8)
    c = torch.stack((c & 15, c >> 4), 2).view(rows, -1)[:, :cols]
    return _values4(c, h["scales"].view(torch.uint8).to(torch.int32)[:, :-(-cols // 32)] - 127)


def _rounded4(x):
    return _values4(*_quantize4(x))


def run(s):
    case = s["case"]
    return (_own if own else _plain)(s, case, case["op"])


def _plain(s, case, op):
    if op == "norm":
        h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
        v = h.float()
        r = torch.rsqrt(v.square().mean(1) + EPS)
        y = v * r[:, None] * s["w"]
        got = {"r": r}
        if s["res"] is not None:
            got["h"] = h
        if case["forms"] == "none":
            got["y"] = y.to(h.dtype)
        if case["forms"] in ("plain", "both"):
            got["plain"] = _quantize8(y)
        if case["forms"] in ("transposed", "both"):
            got["transposed"] = _quantize8(y.t())
        return got
    if op == "norm gradient":
        dy, n = s["dy"].float(), s["x"].float() * s["r"][:, None]
        g = dy * s["w"]
        dh = (g - n * (g * n).mean(1, keepdim=True)) * s["r"][:, None]
        if s["dres"] is not None:
            dh = dh + s["dres"].float()
        return {"dh": dh.to(s["x"].dtype), "dw": (dy * n).sum(0)}
    if op == "embedding":
        ids = s["ids"]
        out = s["table"][ids.clamp_min(0)].float() * math.sqrt(case["cols"])
        if case["pad"]:
            out = out * (ids >= 0)[:, None]
        return out.to(DTYPES[case["dtype"]])
    if op == "embedding gradient":
        g, ids, dy = s["g"], s["ids"], s["dy"].float() * math.sqrt(case["cols"])
        if case["pad"]:
            ids, dy = ids.clamp_min(0), dy * (ids >= 0)[:, None]
        if not case["add"]:
            g.zero_()
        return g.index_add_(0, ids, dy)
    if op == "values":
        got = {}
        if case["forms"] != "transposed":
            got["plain"] = _rounded4(s["x"]).to(torch.bfloat16)
        if case["forms"] != "plain":
            got["transposed"] = _rounded4(s["x"].t()).to(torch.bfloat16)
        return got
    if op == "linear":
        return (_rounded4(s["x"]) @ _values(s["w"]).t()).to(torch.bfloat16)
    if op == "product":
        c = _values(s["a"]) @ _values(s["b"]).t()
        if case["add"]:
            s["c"].copy_(s["c"].float() + c)
            return s["c"]
        return c.to(DTYPES[case["dtype"]])
    x, dy = s["x"], s["dy"]
    y = _rounded4(x) @ _values(s["w"]).t()
    dx = _rounded4(dy) @ _values(s["wt"]).t()
    s["g"].add_(_rounded4(dy.t()) @ _rounded4(x.t()).t())
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "g": s["g"]}


def _view8(q):
    return {"codes": q.codes[:, :q.shape[1]], "scales": q.scales[:, :-(-q.shape[1] // 128)]}


def _own(s, case, op):
    import orthogonalized_updates_amd as mh

    def matrix(h):
        return mh.Fp4Matrix(h["codes"], h["scales"], h["shape"])

    if op == "norm":
        if case["forms"] == "none":
            y, h, r = mh.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS)
            got = {"r": r, "y": y}
        else:
            q, qt, h, r = mh.rms_norm_fp8(s["x"], s["w"], residual=s["res"], eps=EPS, forms=case["forms"])
            got = {"r": r}
            if q is not None:
                got["plain"] = _view8(q)
            if qt is not None:
                got["transposed"] = _view8(qt)
        if s["res"] is not None:
            got["h"] = h
        return got
    if op == "norm gradient":
        dh, dw = mh.rms_norm_backward(s["dy"], s["x"], s["w"], s["r"], dresidual=s["dres"])
        return {"dh": dh, "dw": dw}
    if op == "embedding":
        return mh.embedding(s["ids"], s["table"], scale=math.sqrt(case["cols"]), out_dtype=DTYPES[case["dtype"]])
    if op == "embedding gradient":
        return mh.embedding_backward(s["ids"], s["dy"], s["g"], scale=math.sqrt(case["cols"]), accumulate=case["add"])
    if op == "values":
        q, qt = mh.fp4_quantize(s["x"], forms=case["forms"])
        got = {} if q is None else {"plain": q.dequantize(torch.bfloat16)}
        return got if qt is None else dict(got, transposed=qt.dequantize(torch.bfloat16))
    if op == "linear":
        return mh.fp4_matmul(mh.fp4_quantize(s["x"])[0], matrix(s["w"]))
    if op == "product":
        if case["add"]:
            return mh.fp4_matmul(matrix(s["a"]), matrix(s["b"]), out=s["c"], accumulate=True)
        return mh.fp4_matmul(matrix(s["a"]), matrix(s["b"]), out_dtype=DTYPES[case["dtype"]])
    x, xt = mh.fp4_quantize(s["x"], forms="both")
    dy, dyt = mh.fp4_quantize(s["dy"], forms="both")
    y = mh.fp4_matmul(x, matrix(s["w"]))
    dx = mh.fp4_matmul(dy, matrix(s["wt"]))
    mh.fp4_matmul(dyt, xt, out=s["g"], accumulate=True)
    return {"y": y, "dx": dx, "g": s["g"]}


# ---- from the definition, in 64 bits ----------------------------------------
def _two(e):
    """Exact powers of two: 1 scaled by numpy's ldexp through a table."""
    table = torch.from_numpy(np.ldexp(1.0, np.arange(-160, 161))).to(e.device)
    return table[(e + 160).long()]


def _blocks(x, block, most):
    """x in blocks of a row, padded with zeros, and each block's smallest scale that holds it under `most`."""
    p = torch.nn.functional.pad(x, (0, -x.shape[1] % block)).reshape(x.shape[0], -1, block)
    a = p.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / most))
    e = torch.where(a > most * _two(e), e + 1, e)
    e = torch.where(a <= most * _two(e - 1), e - 1, e)
    return p, _two(torch.where(a > 0, e, torch.full_like(e, -126.0)).clamp_min(-126.0))


def _grid(v, bits, lowest):
    """v rounded to `bits` mantissa bits from 2^lowest up, equal steps below; halves to even."""
    size = v.abs()
    top = torch.floor(torch.log2(torch.where(size > 0, size, torch.ones_like(size))))
    top = torch.where(_two(top) > size, top - 1, top)  # log2 rounded up past a power of two
    top = torch.where(_two(top + 1) <= size, top + 1, top)
    step = _two(top.clamp_min(float(lowest)) - bits)
    return torch.round(v / step) * step


def _exact8(x):
    p, scale = _blocks(x.double(), 128, 448.0)
    return {"codes": _grid(p / scale, 3, -6).reshape(x.shape[0], -1)[:, :x.shape[1]], "scales": scale[:, :, 0]}


def _exact4(x):
    p, scale = _blocks(x.double(), 32, 6.0)
    return (_grid(p / scale, 1, 0) * scale).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _exact_values(h):
    """Codes and scale bytes read bit by bit."""
    rows, cols = h["shape"]
    j = torch.arange(cols, device="cuda")
    c = h["codes"].view(torch.uint8).long()[:, j // 2] >> 4 * (j % 2) & 15
    mant, ex = (c & 1).double(), (c >> 1 & 3).double()
    size = torch.where(ex > 0, (2 + mant) * _two(ex - 2), mant * 0.5)
    return torch.where(c >= 8, -size, size) * _two(h["scales"].view(torch.uint8).double() - 127)[:, j // 32]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    times = lambda a, b: torch.matmul(a, b.t().contiguous())  # noqa: E731
    if op == "norm":
        h = s["x"].double()
        if s["res"] is not None:  # fp32 holds the sum of two bf16 values but for far smaller ones; the definition rounds it
            h = (h + s["res"].double()).to(s["x"].dtype).double()
        r = 1 / torch.sqrt((h * h).sum(1) / case["cols"] + EPS)
        y = h * r.unsqueeze(1) * s["w"].double()
        got = {"r": r}
        if s["res"] is not None:
            got["h"] = h
        if case["forms"] == "none":
            got["y"] = y
        if case["forms"] in ("plain", "both"):
            got["plain"] = _exact8(y)
        if case["forms"] in ("transposed", "both"):
            got["transposed"] = _exact8(y.t())
        return got
    if op == "norm gradient":
        h, r, dy = s["x"].double(), s["r"].double().unsqueeze(1), s["dy"].double()
        g = dy * s["w"].double()
        dot = (g * h).sum(1, keepdim=True)
        dh = g * r - h * r ** 3 * dot / case["cols"]
        return {"dh": dh if s["dres"] is None else dh + s["dres"].double(), "dw": torch.einsum("tc,tc->c", dy, h * r)}
    if op == "embedding":
        ids = s["ids"]
        rows = s["table"].index_select(0, ids.clamp_min(0)).double() * math.sqrt(case["cols"])
        return torch.where((ids >= 0).unsqueeze(1), rows, torch.zeros_like(rows))
    if op == "embedding gradient":
        keep = s["ids"] >= 0
        ids, dy = s["ids"][keep], s["dy"].double()[keep]
        order = torch.argsort(ids, stable=True)
        rows, counts = torch.unique_consecutive(ids[order], return_counts=True)
        sums = torch.segment_reduce(dy[order], "sum", lengths=counts, axis=0) * math.sqrt(case["cols"])
        g = s["g"].double() if case["add"] else torch.zeros(s["g"].shape, device="cuda", dtype=torch.float64)
        g[rows] += sums
        return g
    if op == "values":
        got = {}
        if case["forms"] != "transposed":
            got["plain"] = _exact4(s["x"])
        if case["forms"] != "plain":
            got["transposed"] = _exact4(s["x"].t())
        return got
    if op == "linear":
        return times(_exact4(s["x"]), _exact_values(s["w"]))
    if op == "product":
        c = times(_exact_values(s["a"]), _exact_values(s["b"]))
        return c + s["c"].double() if case["add"] else c
    x, dy = s["x"], s["dy"]
    return {"y": times(_exact4(x), _exact_values(s["w"])), "dx": times(_exact4(dy), _exact_values(s["wt"])),
            "g": s["g"].double() + times(_exact4(dy.t()), _exact4(x.t()))}
