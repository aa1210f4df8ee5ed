"""Plain numpy definitions of the 8-bit floating-point blocks and their products, in 64 bits.
Shares no code with the library."""
import numpy as np

BLOCK = 128
TOP = {"e4m3": 8, "e5m2": 15}                 # exponent of the largest value, 1.75 * 2^TOP


def up(n, to=BLOCK):
    return -(-n // to) * to


def table(kind):
    """The 128 values of codes 0..127 (NaN where the format has no finite value)."""
    exp_bits, frac_bits, bias = (4, 3, 7) if kind == "e4m3" else (5, 2, 15)
    out = np.empty(128)
    for c in range(128):
        e, f = c >> frac_bits, c & ((1 << frac_bits) - 1)
        out[c] = np.ldexp(f, 1 - bias - frac_bits) if e == 0 else np.ldexp((1 << frac_bits) + f, e - bias - frac_bits)
        if (kind == "e4m3" and c == 127) or (kind == "e5m2" and e == 31):
            out[c] = np.nan
    return out


def decode(codes, kind):
    t = table(kind)
    c = codes.astype(np.int64)
    return np.where(c >= 128, -t[c & 127], t[c & 127])


def encode(x, kind):
    """Nearest code, ties to the even one; |x| at most the largest value."""
    t = table(kind)
    t = t[np.isfinite(t)]
    mag = np.abs(x)
    hi = np.clip(np.searchsorted(t, mag), 1, t.size - 1)
    lo = hi - 1
    below, above = mag - t[lo], t[hi] - mag               # exact: neighbours and x have few bits
    code = np.where(below < above, lo, np.where(below > above, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quant(x, kind, tile=False):
    """(codes [rows, 128 * kb], scales [., kb4], blocks with a value that is not finite) of float64 x along its rows."""
    rows, cols = x.shape
    high = BLOCK if tile else 1
    full = np.zeros((up(rows, high), up(cols)))
    full[:rows, :cols] = x
    b = full.reshape(-1, high, full.shape[1] // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all((1, 3))
    most = np.where(np.isfinite(b), np.abs(b), 0).max((1, 3))
    byte = np.zeros(most.shape, np.int64)
    for e in range(255):                                  # the smallest that holds the block
        byte = np.where(most > 1.75 * np.ldexp(1.0, TOP[kind] + e - 127), e + 1, byte)
    unit = np.ldexp(1.0, 127 - byte)[:, None, :, None]
    codes = encode(np.where(np.isfinite(b), b, 0) * unit, kind).reshape(full.shape)[:rows]
    scales = np.zeros((byte.shape[0], up(byte.shape[1], 4)), np.uint8)
    scales[:, :byte.shape[1]] = np.where(bad, 255, byte)
    return codes, scales, bad


def per_element(blocks, rows):
    """What each block has, for each element of [rows, 128 * kb]."""
    out = np.repeat(blocks, BLOCK, 1)
    return out if blocks.shape[0] == rows else np.repeat(out, BLOCK, 0)[:rows]


def values(codes, scales, kind):
    kb = codes.shape[1] // BLOCK
    return decode(codes, kind) * np.ldexp(1.0, per_element(scales[:, :kb].astype(np.int64), codes.shape[0]) - 127)
