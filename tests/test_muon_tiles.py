"""Newton-Schulz and the Muon step in every tile of their products, at sizes that select it, each result's error also
as a root mean square; matrices whose roundings add up."""
import pytest
import torch

import block_quantized_communication_amd as zpq
from test_muon import DT, HALF, close, expected, iterate, make, matrix

pytestmark = pytest.mark.gpu

# tiles of X' and of A
TILES = [(2047, 2050),           # 128; 64 with two buffers
         (2050, 2047),
         (1024, 4096),           # 128; 256, its sums in pieces
         (4095, 1030),
         (2901, 3099),           # 256; 128
         (4500, 4600)]           # 256; 256


@pytest.mark.parametrize("kind", ["plain", "strong", "rank"])
@pytest.mark.parametrize("rows,cols", TILES)
def test_orthogonalize(rows, cols, kind):
    x = matrix(rows, cols, kind, 7)
    close(zpq.orthogonalize(x, out_dtype=torch.float16), iterate(x), HALF["f16"])


@pytest.mark.parametrize("count,rows,cols", [(12, 250, 1000), (10, 1000, 250)])
def test_orthogonalize_batch(count, rows, cols):
    """X' in tiles of 64 with two buffers."""
    x = matrix(rows, cols, "strong", 8, count)
    got = zpq.orthogonalize(x, out_dtype=torch.float16)
    for i in range(count):
        close(got[i], iterate(x[i]), HALF["f16"])


def check(opt, t, before, shapes, half=2.0 ** -24):
    """Momenta to four roundings; weights by the iteration's error: under 2^-8 of the update as a root mean square, times 8 for
    a single one, and what rounding a weight adds."""
    opt.step(lr=0.03, grad_scale=0.5)
    for i, (r, c) in enumerate(shapes):
        m, kept, update = expected(before, i, 0.03, 0.95, True, 0.0, 0.2 * max(r, c) ** 0.5, 0.5)
        assert ((t["m"][i].double() - m).abs() <= 4 * 2.0 ** -24 * (before["m"][i].abs() + before["g"][i].abs())).all()
        d, size = t["p"][i].double() - kept - update, update.square().mean().sqrt()
        slack = 3 * 2.0 ** -24 * before["p"][i].abs() + half * (kept + update).abs()
        assert (d.abs() <= 8 * 2.0 ** -8 * size + slack).all()
        assert d.square().mean().sqrt() <= 2.0 ** -8 * size + slack.square().mean().sqrt()
        if t["copy"] is not None:
            assert torch.equal(t["copy"][i], t["p"][i].to(t["copy"][i].dtype))


# tile of X', or of A
SETS = {"128": [(2047, 2050)], "A in 128": [(1500, 1600), (1500, 1700), (1600, 1500), (1490, 1555)], "128, tall": [(2050, 2047)], "256": [(2901, 3099)],
        "64 with two buffers": [(750, 250), (250, 250), (1000, 250), (250, 1000)] * 3,
        "64 with four": [(750, 250), (250, 251)], "one workgroup": [(64, 192), (200, 48), (33, 33)], "a few rows": [(1, 50), (300, 32), (7, 7)],
        "all": [(2047, 2050), (64, 192), (700, 3), (130, 129)]}


@pytest.mark.parametrize("name", list(SETS))
@pytest.mark.parametrize("p,g,copy", [("f32", "bf16", "bf16"), ("bf16", "f32", None)])
def test_muon_step(name, p, g, copy):
    opt, t, before = make(SETS[name], p, g, copy)
    check(opt, t, before, SETS[name], {"f32": 2.0 ** -24, **HALF}[p])


def adverse(rows, cols, kind):
    """Few rows or columns that are not zero, or few different ones: roundings do not average out."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = torch.zeros(rows, cols, device="cuda")
    if kind == "two rows":
        x[:2] = rand(2, cols)
    elif kind == "two alike":
        x[:2] = rand(1, cols) + 0.3 * rand(2, cols)
    elif kind == "two columns":
        x[:, :2] = rand(rows, 2)
    elif kind == "repeated":
        x = (rand(1, cols) + 0.3 * rand(2, cols)).repeat(rows // 2 + 1, 1)[:rows]
    elif kind == "signs":
        x = rand(rows, 1).sign() @ rand(1, cols).sign() + 0.1 * rand(rows, 1).sign() @ rand(1, cols).sign()
    else:
        x += 1
    return x


@pytest.mark.parametrize("kind", ["two rows", "two alike", "two columns", "repeated", "signs", "ones"])
@pytest.mark.parametrize("rows,cols", [(33, 33), (64, 192), (100, 300), (512, 1024), (2048, 2047)])
def test_adverse_matrices(rows, cols, kind):
    """The same bound as of others, 2^-8 as a root mean square, and half a step of the result."""
    x = adverse(rows, cols, kind)
    want = iterate(x)
    for out in HALF:
        d = zpq.orthogonalize(x, out_dtype=DT[out]).double() - want
        assert d.square().mean().sqrt() <= (2.0 ** -8 + HALF[out]) * want.square().mean().sqrt()


def test_captured_step_takes_new_gradients():
    """set_grads between replays of a captured norm and step, eager work of another optimizer beside it."""
    shapes = [(70, 130), (64, 40), (9, 200), (5, 0), (300, 260)]
    opt, t, _ = make(shapes, copy="bf16", lr=0.02)
    twin, u, _ = make(shapes, copy="bf16", lr=0.02)
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        opt.step(sumsq=opt.grad_sumsq(out=total), max_norm=1.0)
    torch.cuda.synchronize()
    twin.step(sumsq=twin.grad_sumsq(), max_norm=1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.grad_sumsq(out=total)
        opt.step(sumsq=total, max_norm=1.0)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for _ in range(4):
        new = [torch.randn(s, generator=gen, device="cuda").mul_(1e-3).bfloat16() for s in shapes]
        opt.set_grads(new)
        twin.set_grads([x.clone() for x in new])
        graph.replay()
        twin.step(sumsq=twin.grad_sumsq(), max_norm=1.0)
        torch.cuda.synchronize()
        for name in ("p", "m", "copy"):
            assert all(torch.equal(a, b) for a, b in zip(t[name], u[name]))
