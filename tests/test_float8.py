"""8-bit floating-point blocks and their products on the GPU, against float8_ref: codes, exponent bytes
and values are equal; products of small whole numbers are equal too (every order of additions gives
them exactly), others within a bound counted from the roundings."""
import numpy as np
import pytest
import torch

import block_quantized_communication_amd as zpq
import float8_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def up8(codes, scales):
    return codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()


def hard(rows, cols, dtype, seed=0):
    """Values that quantizing has trouble with: ties, the largest value and its neighbours, subnormal
    blocks, zeros of both signs, blocks of very different size."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 10.0 ** rng.uniform(-3, 3, (rows, 1))
    grid = np.round(rng.uniform(-32, 32, (rows, cols)) * 2) / 2             # halves of whole steps: ties
    x = np.where(rng.random((rows, cols)) < 0.4, grid * 2.0 ** rng.integers(-6, 6, (rows, 1)), x)
    x = np.where(rng.random((rows, cols)) < 0.05, -0.0, x)
    pick = rng.random((rows, cols)) < 0.02
    x = np.where(pick, rng.choice([448.0, 464.0, 449.0, 447.0, 1.75, 1.8125, 1.751], (rows, cols)), x)
    x[rng.random(rows) < 0.1] = 0
    if dtype == "f32":
        x[rng.random(rows) < 0.1] *= 2.0 ** -140
        x[rng.random(rows) < 0.05] *= 2.0 ** 110
    elif dtype == "bf16":
        x[rng.random(rows) < 0.1] *= 2.0 ** -120
    else:
        x[rng.random(rows) < 0.1] *= 2.0 ** -22
        x = np.clip(x, -60000, 60000)
    return torch.from_numpy(x).to(DT[dtype])


def check_pair(got, x, kind, tile):
    codes, scales = up8(*got)
    want, want_scales, bad = ref.quant(x, kind, tile)
    assert np.array_equal(scales, want_scales)
    nan = ref.per_element(bad, x.shape[0])
    assert np.array_equal(codes[~nan], want[~nan])
    assert not np.isfinite(ref.decode(codes[nan], kind)).any()


SHAPES = [(1, 1), (1, 128), (3, 1000), (127, 129), (128, 128), (130, 257), (300, 640), (520, 1025)]


@pytest.mark.parametrize("kind", list(F8))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quant(rows, cols, dtype, kind):
    x = hard(rows, cols, dtype)
    x64, xd = x.double().numpy(), x.cuda()
    check_pair(zpq.quant_f8(xd, dtype=F8[kind]), x64, kind, False)
    check_pair(zpq.quant_f8(xd, along="cols", dtype=F8[kind]), x64.T, kind, False)
    a, b = zpq.quant_f8(xd, along="both", dtype=F8[kind])
    check_pair(a, x64, kind, False)
    check_pair(b, x64.T, kind, False)
    check_pair(zpq.quant_f8(xd, tile=True, dtype=F8[kind]), x64, kind, True)
    check_pair(zpq.quant_f8(xd, tile=True, along="cols", dtype=F8[kind]), x64.T, kind, True)
    a, b = zpq.quant_f8(xd, tile=True, along="both", dtype=F8[kind])
    check_pair(a, x64, kind, True)
    check_pair(b, x64.T, kind, True)


@pytest.mark.parametrize("dtype", list(DT))
def test_quant_not_finite(dtype):
    """A block with an infinity or NaN is NaN as a whole; its neighbours are as ever."""
    x = hard(200, 520, dtype, 3)
    for r, c, v in ((0, 0, float("inf")), (5, 200, float("nan")), (150, 519, float("-inf"))):
        x[r, c] = v
    for tile in (False, True):
        for kind in F8:
            a, b = zpq.quant_f8(x.cuda(), tile=tile, along="both", dtype=F8[kind])
            check_pair(a, x.double().numpy(), kind, tile)
            check_pair(b, x.double().numpy().T, kind, tile)
            y = zpq.dequant_f8(*a, cols=520, dtype=torch.float32).cpu().numpy()
            assert not np.isfinite(y[0, :128]).any() and not np.isfinite(y[150, 512:]).any()


def test_quant_strided_and_unaligned():
    """Rows that lie apart, a first element at an odd address, outputs given."""
    flat = hard(70, 301, "bf16", 5).cuda()
    x = flat[:, 1:300]
    out = (torch.empty(70, 384, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(70, 4, dtype=torch.uint8, device="cuda"))
    got = zpq.quant_f8(x, out=out)
    assert got[0] is out[0]
    check_pair(got, x.double().cpu().numpy(), "e4m3", False)
    a, b = zpq.quant_f8(x, along="both", tile=True)
    check_pair(a, x.double().cpu().numpy(), "e4m3", True)
    check_pair(b, x.double().cpu().numpy().T, "e4m3", True)


@pytest.mark.parametrize("kind", list(F8))
@pytest.mark.parametrize("dtype", list(DT))
def test_dequant_every_code(kind, dtype):
    """All 256 codes with exponent bytes over the whole range."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(40, 1)
    bytes_ = torch.zeros(40, 4, dtype=torch.uint8)
    bytes_[:, :2] = torch.linspace(0, 254, 40).round().to(torch.uint8)[:, None]
    got = zpq.dequant_f8(codes.cuda().view(F8[kind]), bytes_.cuda(), dtype=DT[dtype]).cpu()
    want = ref.values(codes.numpy(), bytes_.numpy(), kind)
    fine = np.isfinite(want) & (codes.numpy() & 127 != 124 if kind == "e5m2" else True)
    with np.errstate(over="ignore"):
        want32 = torch.from_numpy(want.astype(np.float32)).to(DT[dtype])       # exact in binary32 or beyond its range
    assert torch.equal(got[torch.from_numpy(fine)], want32[torch.from_numpy(fine)])


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dequant_and_transpose(rows, cols):
    x = hard(rows, cols, "f32", 9)
    a, b = zpq.quant_f8(x.cuda(), tile=True, along="both")
    t = zpq.transpose_f8(*a, cols=cols)
    assert torch.equal(t[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(t[1], b[1])
    for pair, c in ((a, cols), (b, rows)):
        codes, scales = up8(*pair)
        full = torch.full((codes.shape[0] + 1, c + 3), 7.0, device="cuda")
        zpq.dequant_f8(*pair, cols=c, out=full[:-1, :c])
        assert torch.equal(full[:-1, :c].cpu().double(), torch.from_numpy(ref.values(codes, scales, "e4m3")[:, :c]))
        assert (full[-1] == 7).all() and (full[:, c:] == 7).all()


def whole(rows, k, kind, tile, seed):
    """Codes of whole numbers in [-4, 4] (column k and later zero) and exponent bytes 127..129."""
    rng = np.random.default_rng(seed)
    v = np.zeros((rows, ref.up(k)))
    v[:, :k] = rng.integers(-4, 5, (rows, k))
    kb = v.shape[1] // 128
    s = np.zeros((ref.up(rows) // 128 if tile else rows, ref.up(kb, 4)), np.uint8)
    s[:, :kb] = rng.integers(127, 130, (s.shape[0], kb))
    pair = torch.from_numpy(v).float().to(F8[kind]).cuda(), torch.from_numpy(s).cuda()
    return pair, torch.from_numpy(ref.values(ref.encode(v, kind), s, kind)).cuda()


# every tile size with its edges, sums of one block to many, split sums
PRODUCTS = [(1, 1, 1), (1, 300, 129), (3, 5, 640), (16, 16, 128), (17, 33, 511), (64, 64, 512), (65, 63, 700), (1, 1000, 5000),
            (128, 130, 384), (129, 4100, 260), (255, 700, 1000), (300, 300, 2000), (1000, 1100, 140), (2600, 5000, 130),
            (2816, 4864, 1100), (4100, 3600, 900), (40, 9000, 300)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("ka,kb,ta,tb", [("e4m3", "e4m3", False, True), ("e5m2", "e4m3", False, False),
                                         ("e4m3", "e5m2", True, False), ("e5m2", "e5m2", True, True)])
def test_matmul_whole_numbers(m, n, k, ka, kb, ta, tb):
    a, av = whole(m, k, ka, ta, 1)
    b, bv = whole(n, k, kb, tb, 2)
    want = av @ bv.t()                                    # below 2^24: every sum is exact
    got = zpq.matmul_f8(a, b, out_dtype=torch.float32)
    assert torch.equal(got.double(), want)
    full = torch.full((m + 2, n + 5), 3.0, device="cuda")
    zpq.matmul_f8(a, b, out=full[1:m + 1, 2:n + 2], accumulate=True)
    assert torch.equal(full[1:m + 1, 2:n + 2].double(), want + 3)
    full[1:m + 1, 2:n + 2] = 3
    assert (full == 3).all()
    for dtype in (torch.float16, torch.bfloat16):
        assert torch.equal(zpq.matmul_f8(a, b, out_dtype=dtype), want.float().to(dtype))


@pytest.mark.parametrize("m,n,k", [(1, 40, 40000), (15, 17, 9000), (16, 1, 20000), (17, 100, 8300), (32, 33, 12800), (33, 32, 12800)])
def test_matmul_few_rows_and_long_sums(m, n, k):
    """Up to 32 rows, sums split over workgroups: whole numbers, below 2^24 (40000 * 16 * 16)."""
    for tile in (False, True):
        a, av = whole(m, k, "e4m3", False, 3)
        b, bv = whole(n, k, "e4m3", tile, 4)
        want = av @ bv.t()
        for dtype in (torch.float32, torch.bfloat16):
            assert torch.equal(zpq.matmul_f8(a, b, out_dtype=dtype), want.float().to(dtype))


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("m,n,k", [(1, 700, 3000), (33, 500, 4000), (300, 700, 1500), (2700, 4900, 600)])
def test_matmul_error(m, n, k, out):
    """float32 results: k roundings of 2^-23 (the matrix core may cut off) of the products' absolute sum. 16-bit ones:
    products cut off 2^-18 below the largest, and the output's rounding."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, generator=gen, device="cuda") * 10 ** (torch.rand(m, 1, generator=gen, device="cuda") * 6 - 3)
    w = torch.randn(n, k, generator=gen, device="cuda")
    a, b = zpq.quant_f8(x, dtype=torch.float8_e5m2), zpq.quant_f8(w, tile=True)
    av = zpq.dequant_f8(*a, dtype=torch.float32).double()
    bv = zpq.dequant_f8(*b, dtype=torch.float32).double()
    want, size = av @ bv.t(), av.abs() @ bv.abs().t()
    got = zpq.matmul_f8(a, b, out_dtype=DT[out]).double()
    fine = want.abs() < 6e4 if out == "f16" else torch.ones_like(want, dtype=torch.bool)
    sums = size * (k * 2.0 ** -23)
    if out != "f32":
        sums = sums + av.abs().amax(1)[:, None] * bv.abs().amax(1)[None, :] * (k * 2.0 ** -18)
    bound = sums + (want.abs() + sums) * HALF[out] + (2.0 ** -25 if out == "f16" else 0)
    assert ((got - want).abs() <= bound)[fine].all()
    # as a whole far nearer: half of the output's roundings, or of a random walk of k of them
    rel = ((got - want)[fine].norm() / want[fine].norm()).item()
    assert rel <= (HALF[out] + 2.0 ** -23 * k ** 0.5 if out == "f32" else HALF[out] + 2.0 ** -15)


@pytest.mark.parametrize("first,last", [(1, 253), (2, 252)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matmul_scale_range(dtype, first, last):
    """Exponent bytes against their opposites: every product of the two scales is 1. Codes are at least 1, so that no
    element is below 2^-126. With byte 253 a code of 4 is 2^128, which is no binary32 number: such an element is
    infinite in float32 results, where elements are multiplied as binary32 numbers (zpq.h)."""
    blocks = last - first + 1
    k = 128 * blocks
    gen = np.random.default_rng(4)
    va, vb = gen.choice([1.0, 2.0, 3.0, -1.0, -4.0], (40, k)), gen.choice([1.0, 2.0, -3.0, 4.0], (50, k))
    s = np.zeros((1, ref.up(blocks, 4)), np.uint8)
    s[0, :blocks] = np.arange(first, last + 1)
    sa, sb = np.repeat(s, 40, 0), np.repeat(np.where(s > 0, 254 - s, 0), 50, 0).astype(np.uint8)
    pair = lambda v, s: (torch.from_numpy(v).float().to(torch.float8_e4m3fn).cuda(), torch.from_numpy(s).cuda())  # noqa: E731
    got = zpq.matmul_f8(pair(va, sa), pair(vb, sb), out_dtype=dtype)
    if dtype == torch.float32 and last == 253:
        over = (np.abs(va[:, -128:]) == 4).any(1)[:, None] | (np.abs(vb[:, :128]) == 4).any(1)[None, :]
        assert over.all() and not got.isfinite().any()
    else:
        assert torch.equal(got.cpu(), torch.from_numpy(va @ vb.T).float().to(dtype))      # whole numbers below 2^24


def test_matmul_empty_and_nan():
    a, b = zpq.quant_f8(torch.randn(5, 300, device="cuda")), zpq.quant_f8(torch.randn(7, 300, device="cuda"))
    none = zpq.quant_f8(torch.randn(0, 300, device="cuda"))
    assert zpq.matmul_f8(none, b).shape == (0, 7) and zpq.matmul_f8(a, none).shape == (5, 0)
    zero = lambda r: (torch.empty(r, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(r, 0, dtype=torch.uint8, device="cuda"))  # noqa: E731
    out = torch.ones(5, 7, device="cuda")
    zpq.matmul_f8(zero(5), zero(7), out=out, accumulate=True)
    assert (out == 1).all()
    zpq.matmul_f8(zero(5), zero(7), out=out)
    assert (out == 0).all()
    x = torch.randn(5, 300, device="cuda")
    x[2, 150] = float("nan")
    y = zpq.matmul_f8(zpq.quant_f8(x), b)
    assert y[2].isnan().all() and y[[0, 1, 3, 4]].isfinite().all()


def test_matmul_repeats_bit_for_bit():
    x, w = torch.randn(70, 9000, device="cuda"), torch.randn(300, 9000, device="cuda")
    a, b = zpq.quant_f8(x), zpq.quant_f8(w)
    first = zpq.matmul_f8(a, b, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(zpq.matmul_f8(a, b, out_dtype=torch.float32), first)
