"""What is measured of the training step's matrix operators: 8-bit floating-point blocks of 128 (quantizing a
tensor along its rows, along its columns and in 128 x 128 tiles), products of such operands, the three
products of a linear layer with the quantizing in front of them, orthogonalising an update by
Newton-Schulz products, and the Muon step that does so for a layer's matrices.

own = False: the operators' plain forms, elementary torch operations in 32 bits.
own = True:  the calls a user makes of the library.

An operand of a product is a pair: codes [rows, 128 * blocks], float8, the columns past the tensor's
own ones zero, and exponent bytes [rows, blocks rounded up to 4] (or one row for each 128 rows: tiles); an
element is code * 2^(byte - 127).  prepare() makes the operands of the products with the plain form on
both sides; only Muon's handle, which a program makes once, is the library's.
"""
import math

import torch

own = False

BLOCK = 128
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}                 # exponent of the largest value, 1.75 * 2^TOP
COEFFS, STEPS = (3.4445, -4.7750, 2.0315), 5
LR, MOMENTUM, DECAY, MAX_NORM = 3e-4, 0.95, 0.1, 1.0


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # A training batch's activations, for the forward product and the weight gradient at once.
        dict(name="quant batch", op="quant", rows=16384, cols=8192, x="bf16", kind="e4m3", form="both"),
        # An fp32 weight of odd sizes in tiles.
        dict(name="quant odd weight", op="quant", rows=4004, cols=1001, x="f32", kind="e4m3", form="tile"),
        # One token through a hidden-8192 layer's QKV matrix: the weight is read once.
        dict(name="product one token", op="product", m=1, n=24576, k=8192, a="e4m3", tile=True, out="bf16", accumulate=False),
        # A ragged batch through an odd layer.
        dict(name="product odd", op="product", m=999, n=4004, k=1001, a="e4m3", tile=True, out="f16", accumulate=False),
        # A training batch through a hidden-8192 layer's output projection.
        dict(name="product batch", op="product", m=16384, n=8192, k=8192, a="e4m3", tile=True, out="bf16", accumulate=False),
        # The weight gradient of an MLP's half over a batch, added to the fp32 gradient of earlier micro-batches.
        dict(name="product gradient", op="product", m=4096, n=8192, k=16384, a="e5m2", tile=False, out="f32", accumulate=True),
        # Forward and backward of one linear layer of odd sizes on a small batch.
        dict(name="linear small odd", op="linear", tokens=300, cols=250, rows=1001, x="bf16"),
        # The same for 8192 tokens through a hidden-4096 layer's first feed-forward matrix.
        dict(name="linear batch", op="linear", tokens=8192, cols=4096, rows=16384, x="bf16"),
        # A toy model's matrices: latency.
        dict(name="ortho small", op="ortho", count=10, rows=64, cols=192, x="f32", out="bf16"),
        # The feed-forward matrix of a hidden-4096 layer.
        dict(name="ortho large", op="ortho", count=1, rows=16384, cols=4096, x="bf16", out="bf16"),
        # Three layers of odd hidden size, fp32 gradients, no copies.
        dict(name="muon odd layers", op="muon", hidden=250, layers=3, g="f32", copy="none"),
        # One hidden-2048 layer: four matrices, 50.3 M elements.
        dict(name="muon layer", op="muon", hidden=2048, layers=1, g="bf16", copy="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over [lo, hi], evenly in its logarithm; half of them multiples of 64."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 and n >= 64 else n


def draw(rng):
    op = rng.choice(["quant", "product", "product", "linear", "ortho", "muon"])
    if op == "quant":
        rows, cols = _size(rng, 1, 16384), _size(rng, 1, 12288)
        return dict(op=op, rows=rows, cols=cols, x=rng.choice(list(DT)), kind=rng.choice(list(F8)),
                    form=rng.choice(["rows", "cols", "both", "tile"]))
    if op == "product":
        m, n = _size(rng, 1, 16384), _size(rng, 1, 24576)
        k = _size(rng, 1, max(1, min(16384, (1 << 40) // (m * n))))
        return dict(op=op, m=m, n=n, k=k, a=rng.choice(list(F8)), tile=rng.random() < 0.5, out=rng.choice(list(DT)),
                    accumulate=rng.random() < 0.4)
    if op == "linear":
        tokens, rows = _size(rng, 1, 8192), _size(rng, 16, 16384)
        cols = _size(rng, 16, max(16, min(8192, (1 << 38) // (tokens * rows))))
        return dict(op=op, tokens=tokens, cols=cols, rows=rows, x=rng.choice(list(DT)))
    if op == "ortho":
        rows, cols = _size(rng, 1, 4096), _size(rng, 1, 8192)
        most = (1 << 37) // (min(rows, cols) ** 2 * max(rows, cols))
        return dict(op=op, count=_log(rng, 1, max(1, min(64, most))), rows=rows, cols=cols, x=rng.choice(list(DT)),
                    out=rng.choice(["f16", "bf16"]))
    hidden = _size(rng, 16, 2048)
    return dict(op=op, hidden=hidden, layers=_log(rng, 1, max(1, min(12, int((2048 / hidden) ** 3)))), g=rng.choice(list(DT)),
                copy=rng.choice(["none", "f16", "bf16"]))


def _shapes(case):
    """The matrices of a transformer layer: QKV, output projection, two feed-forward matrices."""
    h = case["hidden"]
    return [(3 * h, h), (h, h), (4 * h, h), (h, 4 * h)]


def _up(n, to=BLOCK):
    return -(-n // to) * to


def _bytes(t):
    return 4 if t == "f32" else 2


def _ortho_flops(rows, cols):
    """Two symmetric products, of which one half is computed, and a whole one, each step."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (m * m * n + m * m * m + 2 * m * m * n)


def work(case):
    c = case
    if c["op"] == "quant":
        n = c["rows"] * c["cols"]
        copies = 2 if c["form"] == "both" else 1
        scales = n / (BLOCK * BLOCK if c["form"] == "tile" else BLOCK)
        # read once; codes and exponents written, and read again for the values, which are written in 16 bits
        return {"bytes": n * _bytes(c["x"]) + copies * (2 * (n + scales) + 2 * n), "flops": 0}
    if c["op"] == "product":
        out = c["m"] * c["n"] * _bytes(c["out"]) * (2 if c["accumulate"] else 1)
        return {"bytes": (c["m"] + c["n"]) * c["k"] + out, "flops": 2 * c["m"] * c["n"] * c["k"]}
    if c["op"] == "linear":
        t, i, o, b = c["tokens"], c["cols"], c["rows"], _bytes(c["x"])
        # x, dy and the weight's codes read, y and dx written, the fp32 weight gradient read and written
        return {"bytes": 2 * t * (i + o) * b + i * o + 8 * i * o, "flops": 6 * t * i * o}
    if c["op"] == "ortho":
        return {"bytes": c["count"] * c["rows"] * c["cols"] * (_bytes(c["x"]) + 2),
                "flops": c["count"] * _ortho_flops(c["rows"], c["cols"])}
    n = c["layers"] * sum(a * b for a, b in _shapes(c))
    # weights and momenta read and written, the gradient read for its norm and again, the copy written
    return {"bytes": 16 * n + 2 * n * _bytes(c["g"]) + (0 if c["copy"] == "none" else 2 * n),
            "flops": c["layers"] * sum(_ortho_flops(a, b) for a, b in _shapes(c))}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed, role):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + role) % (1 << 62))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, cols, dtype):
    """Unit size, one column in a hundred thirty times as large, tokens of different size."""
    big = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.01, 30.0, 1.0)
    return _randn(gen, rows, cols).mul_(big).mul_(_randn(gen, rows, 1).mul_(0.5).exp_()).to(dtype)


def _gradients(gen, rows, cols, dtype):
    """Output gradients: tokens differ by three orders of magnitude, a few get none."""
    size = 10.0 ** (torch.rand(rows, 1, generator=gen, device="cuda") * 3 - 5)
    size = torch.where(torch.rand(rows, 1, generator=gen, device="cuda") < 0.02, 0.0, size)
    return _randn(gen, rows, cols).mul_(size).to(dtype)


def _update(gen, shape, dtype):
    """A matrix's gradient: noise of different size for each row and column, and four strong directions."""
    count, rows, cols = shape
    noise = _randn(gen, count, rows, cols)
    noise *= _randn(gen, count, rows, 1).mul_(0.5).exp_() * _randn(gen, count, 1, cols).mul_(0.5).exp_()
    strong = _randn(gen, count, rows, 4) @ _randn(gen, count, 4, cols)
    return noise.add_(strong).mul_(1e-4).to(dtype)


def prepare(case, seed):
    c, op = case, case["op"]
    s = dict(case=c)
    if op == "quant":
        gen = _gen(seed, 21)
        make = _gradients if c["kind"] == "e5m2" else _activations
        s["x"] = _randn(gen, c["rows"], c["cols"]).mul_(0.02).to(DT[c["x"]]) if c["form"] == "tile" else make(gen, c["rows"], c["cols"], DT[c["x"]])
    elif op == "product":
        gen = _gen(seed, 22)
        make = _gradients if c["a"] == "e5m2" else _activations
        s["a"] = _pair(make(gen, c["m"], c["k"], torch.bfloat16), c["a"], False)
        s["b"] = _pair(_randn(gen, c["n"], c["k"]).mul_(0.02), "e4m3", c["tile"])
        if c["accumulate"]:
            s["out"] = _randn(gen, c["m"], c["n"]).mul_(1e-2).to(DT[c["out"]])
    elif op == "linear":
        gen = _gen(seed, 23)
        s["x"] = _activations(gen, c["tokens"], c["cols"], DT[c["x"]])
        s["dy"] = _gradients(gen, c["tokens"], c["rows"], DT[c["x"]])
        s["w"] = _pair(_randn(gen, c["rows"], c["cols"]).mul_(0.02), "e4m3", True)
        s["dw"] = _randn(gen, c["rows"], c["cols"]).mul_(1e-2)
    elif op == "ortho":
        s["x"] = _update(_gen(seed, 24), (c["count"], c["rows"], c["cols"]), DT[c["x"]])
    else:
        gen = _gen(seed, 25)
        shapes = [(c["layers"], a, b) for a, b in _shapes(c)]
        s["g"] = [_update(gen, x, DT[c["g"]]) for x in shapes]
        s["m"] = [_update(gen, x, torch.float32).mul_(4.0) for x in shapes]
        s["p"] = [_randn(gen, *x).mul_(0.02) for x in shapes]
        s["copy"] = None if c["copy"] == "none" else [torch.zeros(x, dtype=DT[c["copy"]], device="cuda") for x in shapes]
    if own:
        import block_quantized_communication_amd as zpq
        s["zpq"] = zpq
        if op == "muon":
            each = lambda stacked: [x[i] for x in stacked for i in range(c["layers"])]  # noqa: E731
            s["opt"] = zpq.Muon(each(s["p"]), each(s["g"]), copies=None if s["copy"] is None else each(s["copy"]), lr=LR,
                                momentum=MOMENTUM, weight_decay=DECAY, momenta=each(s["m"]))
    return s


# ------------------------------------------------------------------------------------- plain forms
def _pow2(e):
    """2^e in 64 bits, exactly, e whole numbers."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _blocks(x, tile):
    """x as [row groups, rows of one, column blocks, 128], zero past its ends."""
    rows, cols = x.shape
    high = BLOCK if tile else 1
    x = torch.nn.functional.pad(x.float(), (0, _up(cols) - cols, 0, _up(rows, high) - rows))
    return x.view(x.shape[0] // high, high, x.shape[1] // BLOCK, BLOCK)


def _pair(x, kind, tile):
    """(codes, exponent bytes) of x: the smallest power of two that leaves the block's largest magnitude at most
    1.75 * 2^TOP."""
    b = _blocks(x, tile)
    most = b.abs().amax((1, 3))
    fraction, exponent = torch.frexp(most)                              # in [1/2, 1)
    e = exponent - 1 - TOP[kind] + (fraction > 0.875).int()
    byte = torch.where(most > 0, e + 127, torch.zeros_like(e)).clamp_(min=0)
    y = b * _pow2(127 - byte)[:, None, :, None].float()
    codes = y.to(F8[kind]).view(-1, b.shape[2] * BLOCK)[:x.shape[0]]
    return codes, torch.nn.functional.pad(byte.to(torch.uint8), (0, _up(byte.shape[1], 4) - byte.shape[1]))


def _values(pair, rows, cols):
    """The values that a pair stands for, in 32 bits."""
    codes, byte = pair
    b = codes.float().view(codes.shape[0], -1, BLOCK)
    scale = _pow2(byte[:, :b.shape[1]].int() - 127).float()
    if byte.shape[0] != codes.shape[0]:
        scale = scale.repeat_interleave(BLOCK, 0)[:codes.shape[0]]
    return (b * scale[:, :, None]).view(codes.shape)[:rows, :cols]


def _quant_plain(s):
    c, x = s["case"], s["x"]
    rows, cols = x.shape
    out = {}
    if c["form"] != "cols":
        pair = _pair(x, c["kind"], c["form"] == "tile")
        out["rows"] = _values(pair, rows, cols).bfloat16()
    if c["form"] in ("cols", "both"):
        out["cols"] = _values(_pair(x.t(), c["kind"], False), cols, rows).bfloat16()
    return out


def _product_plain(s):
    c = s["case"]
    y = _values(s["a"], c["m"], c["k"]) @ _values(s["b"], c["n"], c["k"]).t()
    return s["out"].copy_(s["out"].float() + y) if c["accumulate"] else y.to(DT[c["out"]])


def _linear_plain(s):
    c = s["case"]
    t, i, o, dt = c["tokens"], c["cols"], c["rows"], DT[c["x"]]
    w = _values(s["w"], o, i)
    y = _values(_pair(s["x"], "e4m3", False), t, i) @ w.t()
    dx = _values(_pair(s["dy"], "e5m2", False), t, o) @ w
    dw = _values(_pair(s["dy"].t(), "e5m2", False), o, t) @ _values(_pair(s["x"].t(), "e4m3", False), i, t).t()
    return {"y": y.to(dt), "dx": dx.to(dt), "dw": s["dw"].add_(dw)}


def _ortho_plain(x):
    """Five Newton-Schulz steps on matrices [count, rows, cols] of unit norm."""
    wide = x.shape[1] <= x.shape[2]
    x = x.float() if wide else x.float().transpose(1, 2)
    norm = x.square().sum((1, 2), keepdim=True).sqrt()
    x = x / torch.where(norm > 0, norm, 1.0)
    a, b, c = COEFFS
    for _ in range(STEPS):
        q = x @ x.transpose(1, 2)
        x = a * x + (b * q + c * (q @ q)) @ x
    return x if wide else x.transpose(1, 2)


def _muon_plain(s):
    total = sum(g.double().square().sum() for g in s["g"])
    scale = torch.clamp(MAX_NORM / (total.sqrt() + 1e-6), max=1.0).float()
    out = {"sumsq": total.view(1), "p": s["p"], "m": s["m"]}
    for i, (p, g, m) in enumerate(zip(s["p"], s["g"], s["m"])):
        g = g.float() * scale
        m.mul_(MOMENTUM).add_(g)
        o = _ortho_plain(g + MOMENTUM * m)
        p.mul_(1 - LR * DECAY).sub_(o, alpha=LR * 0.2 * math.sqrt(max(p.shape[1:])))
        if s["copy"] is not None:
            s["copy"][i].copy_(p)
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


# --------------------------------------------------------------------------------------------- run
def run(s):
    c, op = s["case"], s["case"]["op"]
    if not own:
        return {"quant": _quant_plain, "product": _product_plain, "linear": _linear_plain,
                "ortho": lambda s: _ortho_plain(s["x"]).to(DT[c["out"]]), "muon": _muon_plain}[op](s)
    zpq = s["zpq"]
    if op == "quant":
        if c["form"] == "both":
            rows, cols = zpq.quant_f8(s["x"], along="both", dtype=F8[c["kind"]])
            return {"rows": zpq.dequant_f8(*rows, cols=c["cols"]), "cols": zpq.dequant_f8(*cols, cols=c["rows"])}
        if c["form"] == "cols":
            return {"cols": zpq.dequant_f8(*zpq.quant_f8(s["x"], along="cols", dtype=F8[c["kind"]]), cols=c["rows"])}
        return {"rows": zpq.dequant_f8(*zpq.quant_f8(s["x"], tile=c["form"] == "tile", dtype=F8[c["kind"]]), cols=c["cols"])}
    if op == "product":
        if c["accumulate"]:
            return zpq.matmul_f8(s["a"], s["b"], out=s["out"], accumulate=True)
        return zpq.matmul_f8(s["a"], s["b"], out_dtype=DT[c["out"]])
    if op == "linear":
        dt = DT[c["x"]]
        x, x_t = zpq.quant_f8(s["x"], along="both")
        y = zpq.matmul_f8(x, s["w"], out_dtype=dt)
        dy, dy_t = zpq.quant_f8(s["dy"], along="both", dtype=torch.float8_e5m2)
        dx = zpq.matmul_f8(dy, zpq.transpose_f8(*s["w"], cols=c["cols"]), out_dtype=dt)
        return {"y": y, "dx": dx, "dw": zpq.matmul_f8(dy_t, x_t, out=s["dw"], accumulate=True)}
    if op == "ortho":
        return zpq.orthogonalize(s["x"], out_dtype=DT[c["out"]])
    total = s["opt"].grad_sumsq()
    s["opt"].step(sumsq=total, max_norm=MAX_NORM)
    out = {"sumsq": total, "p": s["p"], "m": s["m"]}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


# ------------------------------------------------------------------------------------------- exact
def _nearest(x, kind):
    """float64 values with a power-of-two unit in place (block maximum at most 1.75 * 2^TOP) to the format's grid."""
    bits, least = (3, -6) if kind == "e4m3" else (2, -14)
    step = _pow2(torch.frexp(x)[1].clamp(min=least + 1) - 1 - bits)
    return torch.round(x / step) * step


def _exact_blocks(x, kind, tile):
    """x rounded to 8-bit blocks along its rows, in 64 bits: [rows, cols] back."""
    rows, cols = x.shape
    high = BLOCK if tile else 1
    full = torch.zeros(_up(rows, high), _up(cols), dtype=torch.float64, device="cuda")
    full[:rows, :cols] = x
    b = full.reshape(-1, high, full.shape[1] // BLOCK, BLOCK)
    most = b.abs().amax(dim=(1, 3), keepdim=True)
    unit = _pow2(torch.ceil(torch.log2((most / (1.75 * 2.0 ** TOP[kind])).clamp(min=2.0 ** -127))))
    unit = torch.where(most > unit * 1.75 * 2.0 ** TOP[kind], unit * 2, unit)          # a logarithm that fell short
    unit = torch.where((most <= unit * 0.875 * 2.0 ** TOP[kind]) & (unit > 2.0 ** -127), unit / 2, unit)
    return (_nearest(b / unit, kind) * unit).reshape(full.shape)[:rows, :cols]


def _exact_pair(pair, k):
    codes, byte = pair
    n = codes.shape[0]
    row = torch.arange(n, device="cuda") if byte.shape[0] == n else torch.arange(n, device="cuda") // BLOCK
    at = torch.arange(k, device="cuda") // BLOCK
    return codes[:, :k].double() * _pow2(byte[row].long() - 127)[:, at]


def _exact_ortho(x):
    x = x.double()
    turned = x.shape[-2] > x.shape[-1]
    if turned:
        x = x.mT
    size = torch.linalg.matrix_norm(x)
    x = x / torch.where(size == 0, torch.ones_like(size), size)[:, None, None]
    one = torch.eye(x.shape[1], dtype=torch.float64, device="cuda")
    for _ in range(STEPS):
        q = torch.matmul(x, x.mT)
        x = torch.matmul(COEFFS[0] * one + torch.matmul(COEFFS[1] * one + COEFFS[2] * q, q), x)
    return x.mT if turned else x


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "quant":
        x, out = s["x"].double(), {}
        if c["form"] != "cols":
            out["rows"] = _exact_blocks(x, c["kind"], c["form"] == "tile")
        if c["form"] in ("cols", "both"):
            out["cols"] = _exact_blocks(x.mT, c["kind"], False)
        return out
    if op == "product":
        y = torch.matmul(_exact_pair(s["a"], c["k"]), _exact_pair(s["b"], c["k"]).mT)
        return y + s["out"].double() if c["accumulate"] else y
    if op == "linear":
        x, dy, w = s["x"].double(), s["dy"].double(), _exact_pair(s["w"], c["cols"])
        dw = torch.matmul(_exact_blocks(dy.mT, "e5m2", False), _exact_blocks(x.mT, "e4m3", False).mT)
        return {"y": torch.matmul(_exact_blocks(x, "e4m3", False), w.mT), "dx": torch.matmul(_exact_blocks(dy, "e5m2", False), w),
                "dw": s["dw"].double() + dw}
    if op == "ortho":
        return _exact_ortho(s["x"])
    total = sum((g.double() ** 2).sum() for g in s["g"])
    by = min(1.0, MAX_NORM / (math.sqrt(total.item()) + 1e-6))
    out = {"sumsq": total.reshape(1), "p": [], "m": []}
    for p, g, m in zip(s["p"], s["g"], s["m"]):
        m = MOMENTUM * m.double() + by * g.double()
        o = _exact_ortho(by * g.double() + MOMENTUM * m)
        out["m"].append(m)
        out["p"].append(p.double() * (1 - LR * DECAY) - LR * 0.2 * math.sqrt(max(p.shape[1:])) * o)
    if s["copy"] is not None:
        out["copy"] = out["p"]
    return out
