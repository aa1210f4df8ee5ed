"""The matrix operators past 2^31 and 2^32 elements: parts of a large call equal calls on the parts, or the definition."""
import pytest
import torch

import block_quantized_communication_amd as zpq
from test_muon import HALF

pytestmark = pytest.mark.gpu

ROWS, COLS = 66 * 1024 + 37, 64 * 1024 + 100          # 4.4e9 elements


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.bfloat16)


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("tile", [False, True])
def test_quantizing(tile):
    """The last tiles of rows and of columns, by calls on them alone; back to values; turned round."""
    x = randn(ROWS, COLS)
    a, b = zpq.quant_f8(x, along="both", tile=tile)
    last, edge = (ROWS - 300) // 128 * 128, (COLS - 300) // 128 * 128
    high = 128 if tile else 1
    codes, scales = zpq.quant_f8(x[last:], tile=tile)
    assert same((a[0][last:], a[1][last // high:]), (codes, scales))
    assert torch.equal(zpq.dequant_f8(*a, cols=COLS)[last:], zpq.dequant_f8(codes, scales, cols=COLS))
    codes, scales = zpq.quant_f8(x[:, edge:], along="cols", tile=tile)
    assert same((b[0][edge:], b[1][edge // high:]), (codes, scales))
    if tile:
        assert same(zpq.transpose_f8(*a, cols=COLS), b)
    else:
        assert same(zpq.quant_f8(x), a)


def test_product_of_a_large_operand():
    """A of 4.4e9 codes, by its last rows, within what bfloat16 results lose (zpq.h) and their rounding; a binary32 result of
    4.4e9 values."""
    b = zpq.quant_f8(randn(70, COLS, seed=1))
    a = zpq.quant_f8(randn(ROWS, COLS))
    got = zpq.matmul_f8(a, b, out_dtype=torch.bfloat16)
    last = ROWS - 1000
    av, bv = (zpq.dequant_f8(*p, dtype=torch.float32).double() for p in ((a[0][last:].clone(), a[1][last:].clone()), b))
    want, most = av @ bv.t(), [v.abs().view(v.shape[0], -1, 8).amax(2) for v in (av, bv)]
    cut = 7 * 2.0 ** -13 * (most[0] @ most[1].t()) + COLS * 2.0 ** -23 * (av.abs() @ bv.abs().t())
    assert ((got[last:].double() - want).abs() <= cut + 2.0 ** -8 * (want.abs() + cut)).all()
    del a, got
    one, two = (torch.randint(-4, 5, (n, 128), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").float() for n in (ROWS, COLS))
    pair = lambda v: (v.to(torch.float8_e4m3fn), torch.tensor([[127, 0, 0, 0]], dtype=torch.uint8, device="cuda").repeat(v.shape[0], 1))  # noqa: E731
    out = torch.ones(ROWS, COLS, device="cuda")
    zpq.matmul_f8(pair(one), pair(two), out=out, accumulate=True)
    for rows in (slice(0, 300), slice(ROWS // 2, ROWS // 2 + 300), slice(ROWS - 300, ROWS)):
        assert torch.equal(out[rows], one[rows] @ two.t() + 1)             # whole numbers below 2^24


@pytest.mark.parametrize("rows,cols", [(1024, 2200000), (2200000, 1000), (30, 4194304)])
def test_orthogonalize(rows, cols):
    """A long side, 2.2e9 elements in two of them: by the polynomial of the Gram matrix in 64 bits, at both ends and in the
    middle. Against test_muon's bound, 2^-8 of the result's norm as a root mean square, and half a step."""
    x = randn(rows, cols)
    wide = rows <= cols
    part = lambda t, i, n: (t[:, i:i + n] if wide else t[i:i + n].t()).double()  # noqa: E731
    length, step = max(rows, cols), 1 << 17
    q = sum(p @ p.t() for i in range(0, length, step) for p in (part(x, i, step),))
    size = q.trace()
    q = q / size
    one = torch.eye(q.shape[0], dtype=torch.float64, device="cuda")
    poly, gram = one, q
    a, b, c = zpq.NEWTON_SCHULZ
    for _ in range(5):
        s = a * one + b * gram + c * gram @ gram
        poly, gram = s @ poly, s @ gram @ s
    got = zpq.orthogonalize(x, out_dtype=torch.float16)
    for i in (0, length // 2, length - 5000):
        want = poly @ (part(x, i, 5000) / size.sqrt())
        d = part(got, i, 5000) - want
        assert d.square().mean().sqrt() <= (2.0 ** -8 + HALF["f16"]) * want.square().mean().sqrt()


def test_orthogonalize_matrices_that_lie_far_apart():
    """Strides between matrices and rows whose products pass 2^32."""
    wide = torch.zeros(3, 40, 40000000, dtype=torch.float16, device="cuda")
    x = wide[:, :, 39999000:39999800]
    x.copy_(randn(3, 40, 800))
    assert torch.equal(zpq.orthogonalize(x), zpq.orthogonalize(x.contiguous()))
    out = wide[:, :, 100:900]
    zpq.orthogonalize(x.contiguous(), out=out)
    assert torch.equal(out, zpq.orthogonalize(x.contiguous(), out_dtype=torch.float16))
