"""What is measured of the training-step operators: the optimizer step over many tensors (states in 32
or in 8 bits) with the squared gradient norm it clips by, the embedding lookup (from a float table or
straight from the gathered INT8 blocks) and the embedding's gradient by sorted tokens.

own = False: the operators' plain forms, elementary torch operations in 32 bits (64 for the long sums).
own = True:  the calls a user makes of the library.

Optimizer tensors live as a ZeRO partition keeps them: one flat buffer per role, every tensor starting
at a multiple of 256 elements, the gaps zero.  prepare() also builds the library's handles over these
tensors (the optimizer, the tensor list) where the library is measured: a program makes them once.
"""
import math

import numpy as np
import torch

own = False

ROLE_SEED = {"p": 1, "g": 2, "m": 3, "v": 4}
BETAS, EPS, LR, DECAY, MAX_NORM = (0.9, 0.95), 1e-8, 3e-4, 0.1, 1.0
BLOCK = 256                      # elements per 8-bit state block and per INT8 weight block
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One rank's share of a toy model: ten tensors, 14 thousand elements; all latency.
        dict(name="adamw32 small", op="adamw", bits=32, hidden=64, layers=1, shards=4, g="bf16", copy="bf16", step=3),
        # The 1/16 shard of one hidden-8192 layer (the qwZ workload): 50.3 M elements.
        dict(name="adamw32 layer", op="adamw", bits=32, hidden=8192, layers=1, shards=16, g="bf16", copy="bf16", step=1000),
        # 400 tensors of odd sizes, fp32 gradients, weights in fp32 only.
        dict(name="adamw32 many odd", op="adamw", bits=32, hidden=1001, layers=40, shards=7, g="f32", copy="none", step=17),
        # 8-bit states, a small fine-tuning shard of odd sizes.
        dict(name="adamw8 small odd", op="adamw", bits=8, hidden=250, layers=2, shards=3, g="bf16", copy="f16", step=2),
        # 8-bit states, four hidden-8192 layers of a 1/16 shard: 201 M elements.
        dict(name="adamw8 layers", op="adamw", bits=8, hidden=8192, layers=4, shards=16, g="f16", copy="f16", step=5000),
        # Norm of a small gradient: latency.
        dict(name="norm small", op="norm", hidden=64, layers=1, shards=1, g="bf16"),
        # Norm of half of a hidden-12288 layer's gradient: 906 M elements.
        dict(name="norm large", op="norm", hidden=12288, layers=1, shards=2, g="f16"),
        # A few new tokens through the table: latency.
        dict(name="lookup few", op="lookup", tokens=5, rows=50021, dim=8192, table="f16", out="f16"),
        # A training batch straight from the gathered INT8 table.
        dict(name="lookup int8 batch", op="lookup", tokens=16384, rows=32768, dim=8192, table="i8", out="bf16"),
        # Gradient of a toy table.
        dict(name="embgrad small", op="embgrad", tokens=300, rows=1000, dim=64, dy="f32", out="f32", accumulate=False),
        # A training batch: most rows of a vocabulary of odd size get no token.
        dict(name="embgrad batch", op="embgrad", tokens=16384, rows=50021, dim=8192, dy="bf16", out="bf16", accumulate=False),
        # Many tokens added to the fp32 gradient of earlier micro-batches.
        dict(name="embgrad long", op="embgrad", tokens=131072, rows=65536, dim=2048, dy="f16", out="f32", accumulate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "norm", "lookup", "embgrad"])
    if op in ("adamw", "norm"):
        hidden, shards = _log(rng, 48, 8192), _log(rng, 1, 24)
        most = (130e6 if op == "adamw" else 900e6) * shards / (12.1 * hidden * hidden)
        if most < 1:
            shards = int(math.ceil(shards / most))
            most = 1
        layers = min(_log(rng, 1, 40), max(1, int(most)))
        c = dict(op=op, hidden=hidden, layers=layers, shards=shards, g=rng.choice(list(DT)))
        if op == "adamw":
            c.update(bits=rng.choice([8, 32]), copy=rng.choice(["none", "f16", "bf16"]), step=_log(rng, 1, 10000))
        return c
    tokens, rows = _log(rng, 1, 131072), _log(rng, 3, 131072)
    dim = _log(rng, 33, 8192)
    dim = dim // 16 * 16 if rng.random() < 0.6 and dim >= 64 else dim
    dim = max(1, min(dim, (1 << 28) // max(tokens, rows)))
    if op == "lookup":
        return dict(op=op, tokens=tokens, rows=rows, dim=dim, table=rng.choice(["f32", "f16", "bf16", "i8", "i8"]),
                    out=rng.choice(list(DT)))
    return dict(op=op, tokens=tokens, rows=rows, dim=dim, dy=rng.choice(list(DT)), out=rng.choice(list(DT)),
                accumulate=rng.random() < 0.4)


def _sizes(c):
    """(elements, weight decay) of each tensor: a rank's 1/shards of every matrix and vector of a
    transformer layer (QKV, output projection, two feed-forward matrices, their biases, two norms)."""
    h = c["hidden"]
    one = [(3 * h * h, 1), (h * h, 1), (4 * h * h, 1), (4 * h * h, 1), (3 * h, 0), (h, 0), (4 * h, 0), (h, 0), (h, 0), (h, 0)]
    return [(-(-n // c["shards"]), DECAY * w) for n, w in one] * c["layers"]


def _distinct(case):
    """How many different rows the case's ids name, as expected from their distribution."""
    r = np.arange(1, case["rows"] + 1)
    return float(-np.expm1(case["tokens"] * np.log1p(-0.97 * np.minimum(np.log1p(1 / r) / math.log(case["rows"] + 1), 1))).sum())


def work(case):
    if case["op"] in ("adamw", "norm"):
        n = sum(s for s, _ in _sizes(case))
        gb = 4 if case["g"] == "f32" else 2
        if case["op"] == "norm":
            return {"bytes": n * gb, "flops": 2 * n}
        # weights and both moments read and written once, the gradient once (its norm cannot be known
        # before it has been read whole: once more), the copy written; 8-bit states read out as bf16
        state = 16 * n if case["bits"] == 32 else (4 + 2 + 4) * n + 6 * (-(-n // BLOCK))
        return {"bytes": 8 * n + 2 * gb * n + state + (0 if case["copy"] == "none" else 2 * n), "flops": 20 * n}
    t, v, d, hit = case["tokens"], case["rows"], case["dim"], _distinct(case)
    size = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1 + 4 / BLOCK}
    if case["op"] == "lookup":
        return {"bytes": 8 * t + hit * d * size[case["table"]] + t * d * size[case["out"]], "flops": t * d}
    out = 2 * hit if case["accumulate"] else v
    return {"bytes": 8 * t + t * d * size[case["dy"]] + out * d * size[case["out"]], "flops": t * d}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed, role):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + role) % (1 << 62))


def _ids(case, gen):
    """Token ids as text has them: frequencies about 1/rank, 3% of the positions padding (-1)."""
    t, v = case["tokens"], case["rows"]
    u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(v + 1)) - 1).long().clamp_(0, v - 1)
    pad = torch.rand(t, generator=gen, device="cuda") < 0.03
    return torch.where(pad, torch.full_like(ids, -1), ids)


def _nearest8(x, top):
    """Blocks of x rounded to the nearest 8-bit state value with `top` as the largest exponent field:
    (codes without sign, exponent byte per block)."""
    b = x.abs().view(-1, BLOCK)
    e = ((b.amax(1).view(torch.int32) + 0xFFFFF) >> 23).clamp_(min=1)
    y = (b.double() * _pow2(top - e.long())[:, None]).float().view(torch.int32)
    return ((y + 0x7FFFF + ((y >> 20) & 1)) >> 20).view(-1), e.to(torch.uint8)


def prepare(case, seed):
    if case["op"] == "lookup":
        gen, d, n = _gen(seed, 11), case["dim"], case["rows"] * case["dim"]
        s = dict(case=case, ids=_ids(case, gen), scale=math.sqrt(d))
        if case["table"] == "i8":          # a gathered table is whole blocks: the last one is padded
            full = -(-n // BLOCK) * BLOCK
            s["codes"] = torch.randint(-127, 128, (full,), generator=gen, device="cuda", dtype=torch.int8)
            s["scales"] = torch.rand(full // BLOCK, generator=gen, device="cuda") * 1e-3 + 2e-4
        else:
            s["table"] = torch.randn(case["rows"], d, generator=gen, device="cuda").mul_(0.02).to(DT[case["table"]])
        if own:
            import block_quantized_communication_amd as zpq
            s["zpq"] = zpq
        return s
    if case["op"] == "embgrad":
        gen, shape = _gen(seed, 12), (case["rows"], case["dim"])
        s = dict(case=case, ids=_ids(case, gen), scale=math.sqrt(case["dim"]))
        s["dy"] = torch.randn(case["tokens"], case["dim"], generator=gen, device="cuda").mul_(1e-3).to(DT[case["dy"]])
        if case["accumulate"]:
            s["grad"] = torch.randn(shape, generator=gen, device="cuda").mul_(1e-2).to(DT[case["out"]])
        if own:
            import block_quantized_communication_amd as zpq
            s["zpq"] = zpq
        return s
    sizes = [n for n, _ in _sizes(case)]
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    full = at[-1]
    inside = torch.zeros(full, dtype=torch.bool, device="cuda")
    views = lambda flat: [flat[a:a + n] for a, n in zip(at, sizes)]  # noqa: E731
    for x in views(inside):
        x.fill_(True)
    gen = _gen(seed, ROLE_SEED["g"])
    # gradients differ from block to block by up to four orders of magnitude; one block in a hundred gets none
    size = 10.0 ** (torch.rand(full // BLOCK, generator=gen, device="cuda") * 4 - 5)
    size = torch.where(torch.rand(full // BLOCK, generator=gen, device="cuda") < 0.01, 0.0, size)[:, None]
    g = torch.randn(full, generator=gen, device="cuda").view(-1, BLOCK).mul_(size).view(-1).mul_(inside).to(DT[case["g"]])
    s = dict(case=case, g=g, views=views)
    if case["op"] == "norm":
        if own:
            import block_quantized_communication_amd as zpq
            s["list"] = zpq.TensorList(views(g))
            s["zpq"] = zpq
        return s
    s["p"] = torch.randn(full, generator=_gen(seed, ROLE_SEED["p"]), device="cuda").mul_(0.02).mul_(inside)
    m = torch.randn(full, generator=_gen(seed, ROLE_SEED["m"]), device="cuda").view(-1, BLOCK).mul_(size * 0.3).view(-1).mul_(inside)
    v = torch.randn(full, generator=_gen(seed, ROLE_SEED["v"]), device="cuda").exp_().view(-1, BLOCK).mul_(size * size).view(-1).mul_(inside)
    if case["bits"] == 8:
        code, s["m_exp"] = _nearest8(m, 15)
        s["m"] = (code | ((m < 0) & (code > 0)).int() << 7).to(torch.uint8)
        code, s["v_exp"] = _nearest8(v, 31)
        s["v"] = code.to(torch.uint8)
    else:
        s["m"], s["v"] = m, v
    s["copy"] = None if case["copy"] == "none" else torch.zeros(full, dtype=DT[case["copy"]], device="cuda")
    decay = [w for _, w in _sizes(case)]
    per = torch.tensor([-(-n // BLOCK) for n in sizes], device="cuda")
    s["decay"] = torch.repeat_interleave(torch.tensor(decay, dtype=torch.float64, device="cuda"), per)   # of each block
    s["seed"] = seed % 65521
    if own:
        import block_quantized_communication_amd as zpq
        states = dict(exp_avg=views(s["m"]), exp_avg_sq=views(s["v"]))
        if case["bits"] == 8:
            cut = lambda e: [e[a // BLOCK:-(-(a + n) // BLOCK)] for a, n in zip(at, sizes)]  # noqa: E731
            states = dict(exp_avg=list(zip(views(s["m"]), cut(s["m_exp"]))), exp_avg_sq=list(zip(views(s["v"]), cut(s["v_exp"]))))
        s["opt"] = zpq.AdamW(views(s["p"]), views(g), copies=None if s["copy"] is None else views(s["copy"]), lr=LR, betas=BETAS,
                             eps=EPS, weight_decay=decay, state_bits=case["bits"], seed=s["seed"], **states)
        s["zpq"] = zpq
    return s


# ------------------------------------------------------------------------------------- plain forms
M32, M64 = 0xFFFFFFFF, (1 << 64) - 1


def _pow2(e):
    """2^e in 64 bits, e an int64 tensor."""
    return ((e + 1023) << 52).view(torch.float64)


def _key(seed, step):
    z = (seed + step * 0x9E3779B97F4A7C15) & M64
    z = ((z ^ (z >> 31)) * 0xB7E151628AED2A6B) & M64
    z = ((z ^ (z >> 29)) * 0x243F6A8885A308D3) & M64
    return z >> 32


def _random32(n, seed, step):
    """The 32 random bits of elements 0..n-1 for this seed and step."""
    i = torch.arange(n, device="cuda")
    x = ((i & M32) * 0x9E3779B1 + (i >> 32) * 0x85A308D3 + _key(seed, step)) & M32
    x = ((x ^ (x >> 16)) * 0xB7E15163) & M32
    x = ((x ^ (x >> 15)) * 0x243F6A89) & M32
    return x ^ (x >> 16)


def _value8(code, e, top):
    """Values of unsigned state codes in blocks of exponent byte e."""
    y = (code.int() << 20).view(torch.float32).view(-1, BLOCK).double()
    return (y * _pow2(e.long() - top)[:, None]).float().view(-1)


def _code8(x, top, r16):
    """Blocks of x >= 0 rounded up or down by 16 random bits each: (codes, exponent bytes)."""
    b = x.view(-1, BLOCK)
    e = ((b.amax(1).view(torch.int32) + 0xFFFFF) >> 23).clamp_(min=1)
    y = (b.double() * _pow2(top - e.long())[:, None]).float().view(-1)
    return (y.view(torch.int32) + (r16.int() << 4) + 8) >> 20, e.to(torch.uint8)


def _signed8(code, e):
    x = _value8(code & 127, e, 15)
    return torch.where(code > 127, -x, x)


def _norm_plain(s):
    return s["g"].double().square().sum().view(1)


def _adamw_plain(s):
    c = s["case"]
    (b1, b2), t = BETAS, c["step"]
    f32 = lambda x: torch.tensor(x, dtype=torch.float64).float().item()  # noqa: E731
    total = _norm_plain(s)
    coef = torch.clamp(MAX_NORM / (total.sqrt() + 1e-6), max=1.0).float()
    g = s["g"].float() * coef
    if c["bits"] == 8:
        m, v = _signed8(s["m"], s["m_exp"]), _value8(s["v"], s["v_exp"], 31)
    else:
        m, v = s["m"], s["v"]
    m = m * f32(b1) + g * f32(1 - b1)
    v = v * f32(b2) + (g * f32(1 - b2)) * g
    update = m / (v.sqrt() * f32(1 / math.sqrt(1 - b2 ** t)) + f32(EPS))
    p = (s["p"].view(-1, BLOCK) * (1 - LR * s["decay"]).float()[:, None]).view(-1) - update * f32(LR / (1 - b1 ** t))
    out = {"p": s["p"].copy_(p), "sumsq": total}
    if s["copy"] is not None:
        out["copy"] = s["copy"].copy_(p)
    if c["bits"] == 32:
        out["m"], out["v"] = s["m"].copy_(m), s["v"].copy_(v)
        return out
    r = _random32(m.numel(), s["seed"], t)
    code, e = _code8(m.abs(), 15, r & 0xFFFF)
    s["m"].copy_(code | (m < 0).int() << 7)
    s["m_exp"].copy_(e)
    code, e = _code8(v, 31, r >> 16)
    s["v"].copy_(torch.where((code == 0) & (v > 0), 1, code))      # a positive second moment stays positive
    s["v_exp"].copy_(e)
    out["m"] = _signed8(s["m"], s["m_exp"]).bfloat16()
    out["v"] = _value8(s["v"], s["v_exp"], 31).bfloat16()
    return out


def _lookup_plain(s):
    c, ids = s["case"], s["ids"]
    there = (ids >= 0) & (ids < c["rows"])
    at = torch.where(there, ids, 0)
    if c["table"] == "i8":
        n = c["rows"] * c["dim"]
        x = s["codes"][:n].view(c["rows"], c["dim"])[at].float()
        if c["dim"] % BLOCK == 0:
            x.view(ids.numel(), -1, BLOCK).mul_(s["scales"].view(c["rows"], -1)[at][:, :, None])
        else:
            x.mul_(s["scales"][(at[:, None] * c["dim"] + torch.arange(c["dim"], device="cuda")) // BLOCK])
    else:
        x = s["table"][at].float()
    return (x.mul_(s["scale"]) * there[:, None]).to(DT[c["out"]])


def _embgrad_plain(s):
    c, ids = s["case"], s["ids"]
    there = (ids >= 0) & (ids < c["rows"])
    total = torch.zeros(c["rows"], c["dim"], device="cuda")
    total.index_add_(0, torch.where(there, ids, 0), s["dy"].float() * there[:, None])
    total.mul_(s["scale"])
    if c["accumulate"]:
        return s["grad"].copy_(s["grad"].float() + total)
    return total.to(DT[c["out"]])


# --------------------------------------------------------------------------------------------- run
def run(s):
    c = s["case"]
    if not own:
        return {"adamw": _adamw_plain, "norm": _norm_plain, "lookup": _lookup_plain, "embgrad": _embgrad_plain}[c["op"]](s)
    zpq = s["zpq"]
    if c["op"] == "norm":
        return zpq.grad_sumsq(s["list"])
    if c["op"] == "lookup":
        if c["table"] == "i8":
            return zpq.embedding_i8(s["ids"], s["codes"], s["scales"], c["rows"], c["dim"], block=BLOCK, scale=s["scale"],
                                    out_dtype=DT[c["out"]])
        return zpq.embedding(s["ids"], s["table"], scale=s["scale"], out_dtype=DT[c["out"]])
    if c["op"] == "embgrad":
        if c["accumulate"]:
            return zpq.embedding_grad(s["ids"], s["dy"], c["rows"], scale=s["scale"], out=s["grad"], accumulate=True)
        return zpq.embedding_grad(s["ids"], s["dy"], c["rows"], scale=s["scale"], out_dtype=DT[c["out"]])
    total = s["opt"].grad_sumsq()
    s["opt"].step(c["step"], sumsq=total, max_norm=MAX_NORM)
    out = {"p": s["p"], "sumsq": total}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    if c["bits"] == 32:
        out["m"], out["v"] = s["m"], s["v"]
    else:
        out["m"] = zpq.state8_unpack(s["m"], s["m_exp"], moment=1, dtype=torch.bfloat16)
        out["v"] = zpq.state8_unpack(s["v"], s["v_exp"], moment=2, dtype=torch.bfloat16)
    return out


# ------------------------------------------------------------------------------------------- exact
def _exact8(x, fields, r16):
    """x >= 0 to the two neighbouring values of an 8-bit float with 3 fraction bits, the upper one where the
    place between them plus the random number reaches 1; the largest binade is the one that holds the
    block's largest value after rounding up to 3 fraction bits. `fields`: binades, subnormals included."""
    b = x.view(-1, BLOCK)
    fraction, exponent = torch.frexp(b.amax(1, keepdim=True))     # in [1/2, 1)
    top = exponent - 1 + (fraction > 1 - 1 / 16).int()            # over 1.875 of its binade: it rounds up into the next
    top = torch.where(b.amax(1, keepdim=True) == 0, torch.full_like(top, -126), top).clamp(min=-126)
    own_binade = torch.frexp(b)[1] - 1
    step = torch.ldexp(torch.ones_like(b), torch.maximum(own_binade, top - fields + 1) - 3)
    u = (r16.double().view(-1, BLOCK) * 16 + 8) / 2 ** 20
    return (torch.floor(b / step + u) * step), torch.ldexp(torch.ones_like(top, dtype=torch.float64), top - fields + 1 - 3)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return (s["g"].to(torch.float64) ** 2).sum().reshape(1)
    if case["op"] == "lookup":
        ids, d = s["ids"], case["dim"]
        if case["table"] == "i8":
            n = case["rows"] * d
            table = lambda r: (s["codes"][r[:, None] * d + torch.arange(d, device="cuda")].double()  # noqa: E731
                               * s["scales"].double()[(r[:, None] * d + torch.arange(d, device="cuda")) // BLOCK])
        else:
            table = lambda r: s["table"].index_select(0, r).double()  # noqa: E731
        out = torch.zeros(ids.numel(), d, dtype=torch.float64, device="cuda")
        known = torch.nonzero((ids >= 0) & (ids < case["rows"])).view(-1)
        out[known] = table(ids[known]) * s["scale"]
        return out
    if case["op"] == "embgrad":
        known = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["rows"])).view(-1)
        out = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        out.index_put_((s["ids"][known],), s["dy"][known].double() * s["scale"], accumulate=True)
        return out + s["grad"].double() if case["accumulate"] else out
    (b1, b2), t = BETAS, case["step"]
    g = s["g"].double()
    total = (g * g).sum()
    g = g * min(1.0, MAX_NORM / (math.sqrt(total.item()) + 1e-6))
    if case["bits"] == 8:
        code, shift = s["m"].long(), s["m_exp"].long().repeat_interleave(BLOCK)
        f, q = (code >> 3) & 15, code & 7
        m = torch.where(f > 0, 8 + q, q).double() * torch.where(code > 127, -1.0, 1.0)
        m = torch.ldexp(m, (f.clamp(min=1) - 15 + shift - 127 - 3))
        code, shift = s["v"].long(), s["v_exp"].long().repeat_interleave(BLOCK)
        f, q = code >> 3, code & 7
        v = torch.ldexp(torch.where(f > 0, 8 + q, q).double(), (f.clamp(min=1) - 31 + shift - 127 - 3))
    else:
        m, v = s["m"].double(), s["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = s["p"].double()
    decay = s["decay"].repeat_interleave(BLOCK)
    p = p - LR * decay * p - LR * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + EPS)
    out = {"p": p, "sumsq": total.reshape(1), "copy": None if s["copy"] is None else p, "m": m, "v": v}
    if case["bits"] == 8:
        r = _random32(m.numel(), s["seed"], t)
        mag, _ = _exact8(m.abs(), 15, r & 0xFFFF)
        out["m"] = torch.copysign(mag.view(-1), m)
        val, least = _exact8(v, 31, r >> 16)
        out["v"] = torch.where(v.view(-1, BLOCK) > 0, torch.maximum(val, least), val).view(-1)
    if out["copy"] is None:
        del out["copy"]
    return out
