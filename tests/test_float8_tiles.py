"""Products of 8-bit blocks in every tile loop, at sizes that select it, with ragged edges and more than four blocks
along the sum (a word of exponents is taken up again), and with blocks that are not finite."""
import pytest
import torch

import block_quantized_communication_amd as zpq
from test_float8 import DT, F8, whole

pytestmark = pytest.mark.gpu

# size: tile for bf16 results, tile for float32 and float16 ones
SIZES = [(5, 200, 700),          # few rows
         (70, 130, 700),         # 64, four buffers; the same
         (999, 4004, 1001),      # 64, two buffers; 128
         (1500, 1601, 1100),     # 64, two buffers; the same
         (999, 4004, 4100),      # 64, two buffers; 128, the sum in two parts
         (3000, 3300, 700),      # 256; 128
         (2816, 4864, 700)]      # 256; 256


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("ka,kb,ta,tb", [("e4m3", "e4m3", False, True), ("e5m2", "e4m3", False, False),
                                         ("e4m3", "e5m2", True, False), ("e5m2", "e5m2", True, True)])
def test_whole_numbers(m, n, k, ka, kb, ta, tb):
    """Below 2^24, so that every order of additions gives them exactly; the surroundings stay as they were."""
    a, av = whole(m, k, ka, ta, 1)
    b, bv = whole(n, k, kb, tb, 2)
    want = av @ bv.t()
    for dtype in DT.values():
        full = torch.full((m + 2, n + 5), 3.0, dtype=dtype, device="cuda")
        zpq.matmul_f8(a, b, out=full[1:m + 1, 2:n + 2])
        assert torch.equal(full[1:m + 1, 2:n + 2], want.float().to(dtype))
        full[1:m + 1, 2:n + 2] = 3
        zpq.matmul_f8(a, b, out=full[1:m + 1, 2:n + 2], accumulate=True)
        assert torch.equal(full[1:m + 1, 2:n + 2], (want + 3).float().to(dtype))
        full[1:m + 1, 2:n + 2] = 3
        assert (full == 3).all()


@pytest.mark.parametrize("m,n,k", SIZES)
def test_error(m, n, k):
    """float32 results: k roundings of 2^-23 of the products' absolute sum."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, generator=gen, device="cuda") * 10 ** (torch.rand(m, 1, generator=gen, device="cuda") * 6 - 3)
    a = zpq.quant_f8(x, dtype=torch.float8_e5m2)
    b = zpq.quant_f8(torch.randn(n, k, generator=gen, device="cuda"), tile=True)
    av, bv = (zpq.dequant_f8(*p, dtype=torch.float32).double() for p in (a, b))
    got = zpq.matmul_f8(a, b, out_dtype=torch.float32).double()
    assert ((got - av @ bv.t()).abs() <= k * 2.0 ** -23 * (av.abs() @ bv.abs().t())).all()


@pytest.mark.parametrize("kind", list(F8))
@pytest.mark.parametrize("m,n,k", SIZES)
def test_blocks_that_are_not_finite(m, n, k, kind):
    """Rows and columns that such a block belongs to are NaN; the others what they are without it, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    x, w = torch.randn(m, k, generator=gen, device="cuda"), torch.randn(n, k, generator=gen, device="cuda")
    bad = x.clone()
    bad[m // 2, 3], bad[m - 1, k - 1] = float("nan"), float("inf")
    bad_w = w.clone()
    bad_w[n - 1, k // 2] = float("-inf")
    rows = torch.zeros(m, dtype=torch.bool, device="cuda")
    rows[[m // 2, m - 1]] = True
    for tile in (False, True):
        columns = torch.zeros(n, dtype=torch.bool, device="cuda")
        columns[(n - 1) // 128 * 128 if tile else n - 1:] = True
        nan = rows[:, None] | columns[None, :]
        a, b = zpq.quant_f8(bad, dtype=F8[kind]), zpq.quant_f8(bad_w, tile=tile)
        clean = zpq.quant_f8(x, dtype=F8[kind]), zpq.quant_f8(w, tile=tile)
        for dtype in DT.values():
            got, want = zpq.matmul_f8(a, b, out_dtype=dtype), zpq.matmul_f8(*clean, out_dtype=dtype)
            assert torch.equal(got.isnan(), nan)
            assert torch.equal(got[~nan], want[~nan])
