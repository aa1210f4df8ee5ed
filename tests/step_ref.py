"""Plain numpy definitions of the step operators, for the tests: 64-bit
arithmetic where a tolerance is derived, binary32 operation by operation where
codes must be equal.  Shares no code with the library."""
import math

import numpy as np

M64 = (1 << 64) - 1
BLOCK = 256
U = 2.0 ** -24                # half a step of binary32, relative
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}   # half the smallest subnormal, or more
f32 = np.float32


def padded(n):
    return -(-n // BLOCK) * BLOCK


def clip_factor(sumsq, grad_scale, max_norm):
    if sumsq is None:
        return float(f32(grad_scale))
    norm = math.sqrt(sumsq) * grad_scale
    return float(f32(grad_scale * min(1.0, max_norm / (norm + 1e-6))))


def random32(first, n, seed, step):
    z = (seed + step * 0x9E3779B97F4A7C15) & M64
    z = ((z ^ (z >> 31)) * 0xB7E151628AED2A6B) & M64
    z = ((z ^ (z >> 29)) * 0x243F6A8885A308D3) & M64
    i = np.arange(first, first + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        x = ((i & np.uint64(0xFFFFFFFF)) * np.uint64(0x9E3779B1)
             + (i >> np.uint64(32)) * np.uint64(0x85A308D3) + np.uint64(z >> 32)).astype(np.uint32)
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0xB7E15163)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x243F6A89)
    return x ^ (x >> np.uint32(16))


def per_element(exps, n):
    return np.repeat(exps.astype(np.int64), BLOCK)[:n]


def decode8(codes, exps, moment):
    """float64 values from the definition (zpq.h)."""
    c, e = codes.astype(np.int64), per_element(exps, codes.size)
    top = 15 if moment == 1 else 31
    mag = c & 127 if moment == 1 else c
    f, q = mag >> 3, mag & 7
    x = np.ldexp(np.where(f > 0, 8 + q, q) / 8.0, np.maximum(f, 1) - top + e - 127)
    x = np.where((e == 255) & (mag == (127 if moment == 1 else 255)), np.inf, x)
    return np.where(c >= 128, -x, x) if moment == 1 else x


def exponents(x):
    """Exponent byte of each block of binary32 magnitudes."""
    b = np.zeros(padded(x.size), f32)
    b[:x.size] = np.abs(x)
    a = b.view(np.uint32).reshape(-1, BLOCK).max(1).astype(np.int64)
    return np.clip((a + 0xFFFFF) >> 23, 1, 255).astype(np.uint8)


def encode8(x, moment, rnd16=None):
    """(codes, exponents) of binary32 values: by 16 random bits each, or to
    nearest even where rnd16 is None.  Places between the two neighbours are
    worked out in 64 bits."""
    e8 = exponents(x)
    e = per_element(e8, x.size)
    top = 15 if moment == 1 else 31
    with np.errstate(invalid="ignore", over="ignore"):
        # magnitudes with the block's top binade moved to exponent field `top`, as binary32
        y = np.ldexp(np.abs(x.astype(np.float64)), top - e).astype(f32)
        field = np.where(y > 0, np.maximum(np.frexp(y)[1] + 126, 1), 1)   # binary32 exponent field, subnormals as 1
        place = np.ldexp(y.astype(np.float64), 127 - field + 3)   # in steps; 8..16, below 8 for subnormals
        if rnd16 is None:
            k = np.rint(place)
        else:
            k = np.floor(place + (rnd16.astype(np.float64) * 16 + 8) / 2 ** 20)
        k = np.where(np.isfinite(k), k, 0).astype(np.int64)
    c = k + (field - 1) * 8                                   # a carry moves into the next field by itself
    if moment == 2 and rnd16 is not None:
        c = np.where((c == 0) & (x > 0), 1, c)
    if moment == 1:
        c = c | np.signbit(x).astype(np.int64) << 7
    c = np.where(e == 255, 127 if moment == 1 else 255, c)
    return c.astype(np.uint8), e8


def adamw64(p, g, m, v, c, lr, betas, eps, decay, step):
    """One step in 64 bits from float64 inputs: (p, m, v) and, for each, how far a
    binary32 evaluation in the order of zpq.h may be off: U for every rounding
    of a term or a constant in it, the root within 1 ulp, the quotient as a
    1-ulp reciprocal and a product."""
    b1, b2 = betas
    x = g * c
    m1 = b1 * m + (1 - b1) * x
    mm = np.abs(b1 * m) + np.abs((1 - b1) * x)
    v1 = b2 * v + (1 - b2) * x * x
    root = np.sqrt(v1) / math.sqrt(1 - b2 ** step)
    den = root + eps
    rate = lr / (1 - b1 ** step)
    p1 = p * (1 - lr * decay) - rate * m1 / den
    tm = 6 * U * mm + 2e-45          # m: constant, product, sum; g: c, g*c, constant, product, sum
    tv = 9 * U * v1 + 2e-45          # g'^2: c and g*c twice, constant, two products, sum
    # den: half of v's 9, root 2, constant 1, product 1, sum 1, eps 1; then reciprocal 2, product 1
    tp = U * (4 * np.abs(p) + rate / den * (7 * mm + 18 * np.abs(m1))) + 2e-45
    return p1, m1, v1, tp, tm, tv


def adamw32_moments(g, m, v, c, betas):
    """The new moments in binary32, operation by operation."""
    b1, o1 = f32(betas[0]), f32(1 - betas[0])
    b2, o2 = f32(betas[1]), f32(1 - betas[1])
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        x = g.astype(f32) * f32(c)
        return m.astype(f32) * b1 + x * o1, v.astype(f32) * b2 + (x * o2) * x


def lookup64(ids, table, scale, first=0):
    """float64 rows; table float64 [rows, dim]."""
    out = np.zeros((ids.size, table.shape[1]))
    r = ids.astype(object) - first
    there = np.array([0 <= x < table.shape[0] for x in r], bool)
    at = np.array([int(x) if ok else 0 for x, ok in zip(r, there)], np.int64)
    out[there] = table[at[there]] * scale
    return out


def grad64(ids, dy, rows, scale, first=0, padding=None):
    """(gradient, sum of magnitudes, terms per row) in 64 bits."""
    g = np.zeros((rows, dy.shape[1]))
    mag = np.zeros_like(g)
    n = np.zeros(rows, np.int64)
    r = ids - first
    there = (r >= 0) & (r < rows)
    if padding is not None:
        there &= ids != padding
    np.add.at(g, r[there], dy[there])
    np.add.at(mag, r[there], np.abs(dy[there]))
    np.add.at(n, r[there], 1)
    return g * scale, mag * abs(scale), n
