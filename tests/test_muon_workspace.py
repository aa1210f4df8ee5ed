"""The workspace of orthogonalising and of a Muon plan is bounded, whatever the number of matrices, and many small
ones go through it in several groups."""
import ctypes

import pytest
import torch

import block_quantized_communication_amd as zpq

TABLE = lambda count: 248 * count + 64 + 256  # noqa: E731
BOUND = (1 << 30) + (1 << 29)                # zpq.h: a group's room, and parts of long sums


@pytest.mark.parametrize("count,rows,cols", [(1 << 20, 1, 1), (1 << 18, 1, 256), (1 << 20, 3, 20), (1 << 17, 32, 33), (15000, 65, 65),
                                             (1 << 20, 5, 5), (1000, 1024, 1024), (1 << 16, 33, 300), (1, 6057, 10784)])
def test_orthogonalize(count, rows, cols):
    need = ctypes.c_int64()
    assert zpq.lib().zpq_orthogonalize_bytes(count, rows, cols, ctypes.byref(need)) == 0
    assert need.value <= TABLE(count) + BOUND


@pytest.mark.parametrize("rows,cols,each", [(4096, 4096, 14.1), (1024, 1024, 14.1), (1 << 12, 1 << 14, 14.1), (32, 1 << 20, 5.1), (1, 1 << 22, 36.1)])
def test_bytes_of_an_element(rows, cols, each):
    """What the documentation says of one matrix."""
    need = ctypes.c_int64()
    assert zpq.lib().zpq_orthogonalize_bytes(1, rows, cols, ctypes.byref(need)) == 0
    assert need.value <= TABLE(1) + each * rows * cols


@pytest.mark.parametrize("rows,cols,pieces", [(4096, 16384, 3), (4096, 8192, 0), (2043, 3411, 0), (498, 3061, 0)])
def test_pieces_are_worth_their_memory(rows, cols, pieces):
    """Room for at most so many parts of A's sums, binary32 in 256 x 256 tiles on and under the diagonal, beside X, its
    three copies in 16 bits, A and B: sides to 64, and 64 KB of the rest."""
    up = lambda n: -(-n // 64) * 64  # noqa: E731
    need, t = ctypes.c_int64(), -(-rows // 256)
    assert zpq.lib().zpq_orthogonalize_bytes(1, rows, cols, ctypes.byref(need)) == 0
    room = rows * cols * 4 + rows * up(cols) * 2 + 2 * cols * up(rows) * 2 + 2 * rows * up(rows) * 2
    assert need.value <= room + rows * cols // 256 + 65536 + pieces * t * (t + 1) // 2 * (256 * 256 * 4)


def test_plan():
    need = ctypes.c_int64()
    for shapes in ([(1 + i % 7, 1 + i % 5) for i in range(200000)], [(1, 0)] * 1000 + [(2, 3)] * 150000):
        rows = (zpq._MuonMatrix * len(shapes))()
        for r, (r.rows, r.cols) in zip(rows, shapes):
            pass
        assert zpq.lib().zpq_muon_plan_bytes(rows, len(shapes), ctypes.byref(need)) == 0
        assert need.value <= TABLE(len(shapes)) + BOUND


@pytest.mark.gpu
def test_more_small_matrices_than_fit():
    """90,000 of 3 x 4 take 13 KB each: two groups. Against the iteration in 64 bits. Sides this small go by one small
    matrix in 64 bits, of norm 485 at most (3.4445^5: what a small singular value grows by), times X, of norm 1; both are
    rounded to 24 bits, and so are a sum's three products and two additions: under 500 * 8 * 2^-24, and half a step."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(90000, 3, 4, generator=gen, device="cuda")
    got = zpq.orthogonalize(x, out_dtype=torch.float16).double()
    y = x.double()
    y = y / y.square().sum((1, 2), keepdim=True).sqrt()
    a, b, c = zpq.NEWTON_SCHULZ
    for _ in range(5):
        q = y @ y.mT.contiguous()
        y = a * y + (b * q + c * q @ q) @ y
    assert ((got - y).abs() <= 2.0 ** -11 * y.abs() + 500 * 8 * 2.0 ** -24).all()
