"""Newton-Schulz orthogonalisation and the Muon step on the GPU against the iteration in 64 bits.

Tolerances: operands are rounded to 11 bits (2^-12 of each on average, A, B and X, independent), and X itself is
binary32, so an iteration adds at most about 3 * 2^-12 of the result's norm and five of them, of which the later ones
shrink what the earlier added, under 2^-8 together; the output adds half a step of its type. Single values are off by
that norm spread evenly, times 8 for the largest of a million."""
import numpy as np
import pytest
import torch

import block_quantized_communication_amd as zpq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TRIPLE = (3.4445, -4.7750, 2.0315)


def iterate(x, coeffs=(TRIPLE,) * 5):
    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    size = x.square().sum((-2, -1), keepdim=True).sqrt()
    x = x / torch.where(size == 0, 1.0, size)
    for a, b, c in coeffs:
        q = x @ x.mT
        x = a * x + (b * q + c * q @ q) @ x
    return x.mT if tall else x


def close(got, want, half, most=2.0 ** -8):
    got, size = got.double(), want.square().mean().sqrt()
    d = got - want
    assert d.square().mean().sqrt() <= (most + half) * size
    assert (d.abs() <= 8 * most * size + half * want.abs()).all()


def matrix(rows, cols, kind="plain", seed=0, count=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (rows, cols) if count is None else (count, rows, cols)
    x = torch.randn(*shape, generator=gen, device="cuda")
    if kind == "strong":                                       # a few large singular values over a floor
        x = x * 0.05 + torch.randn(*shape[:-1], 4, generator=gen, device="cuda") @ torch.randn(*shape[:-2], 4, cols, generator=gen, device="cuda")
    elif kind == "rank":                                       # rank 3, if it has as many
        x = torch.randn(*shape[:-1], 3, generator=gen, device="cuda") @ torch.randn(*shape[:-2], 3, cols, generator=gen, device="cuda")
    return x


SHAPES = [(1, 1), (1, 64), (64, 1), (2, 300), (63, 65), (64, 64), (65, 63), (128, 500), (500, 128), (129, 257), (300, 300), (700, 300),
          (1030, 2100), (2100, 1030), (64, 20000), (20000, 70), (1, 5000)]


@pytest.mark.parametrize("kind", ["plain", "strong", "rank"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols, kind):
    x = matrix(rows, cols, kind)
    want = iterate(x)
    for out in HALF:
        close(zpq.orthogonalize(x, out_dtype=DT[out]), want, HALF[out])


@pytest.mark.parametrize("rows,cols", [(33, 33), (33, 256), (256, 40), (48, 47), (64, 256), (256, 64), (64, 257), (32, 33), (50, 200)])
def test_orthogonalize_one_workgroup(rows, cols):
    """Sizes at and around what one workgroup takes, each in every orientation."""
    for kind in ("plain", "strong", "rank"):
        x = matrix(rows, cols, kind, 11)
        for out in HALF:
            close(zpq.orthogonalize(x, out_dtype=DT[out]), iterate(x), HALF[out])


@pytest.mark.parametrize("rows,cols", [(2048, 9000), (3700, 3650), (5000, 5100)])
def test_orthogonalize_large(rows, cols):
    x = matrix(rows, cols, "strong").bfloat16()
    close(zpq.orthogonalize(x, out_dtype=torch.float16), iterate(x), HALF["f16"])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("count,rows,cols", [(3, 100, 60), (50, 64, 192), (2, 700, 650), (25, 10, 9), (7, 130, 128)])
def test_orthogonalize_batch(count, rows, cols, dtype):
    x = matrix(rows, cols, "strong", 1, count).to(DT[dtype])
    got = zpq.orthogonalize(x)
    for i in range(count):
        close(got[i], iterate(x[i]), HALF["bf16"])


def test_orthogonalize_strides():
    """Rows and matrices that lie apart, odd addresses, an output that is part of another tensor."""
    wide = matrix(90, 403, "plain", 2, 3).half()
    x = wide[:, 5:80, 1:400]
    full = torch.full((3, 80, 450), 5.0, dtype=torch.bfloat16, device="cuda")
    got = zpq.orthogonalize(x, out=full[:, 2:77, 3:402])
    for i in range(3):
        close(got[i], iterate(x[i]), HALF["bf16"])
    full[:, 2:77, 3:402] = 5
    assert (full == 5).all()


def test_orthogonalize_steps_and_coeffs():
    x = matrix(90, 200, "strong", 3)
    for steps in (1, 2, 3, 8):
        close(zpq.orthogonalize(x, steps=steps, out_dtype=torch.float16), iterate(x, (TRIPLE,) * steps), HALF["f16"])
    own = ((4.0, -6.0, 3.0), (3.0, -4.0, 2.0), (1.5, -0.5, 0.0))
    close(zpq.orthogonalize(x, steps=3, coeffs=own, out_dtype=torch.float16), iterate(x, own), HALF["f16"])


def test_orthogonalize_edges():
    z = torch.zeros(2, 70, 90, device="cuda")
    z[1] = matrix(70, 90)
    got = zpq.orthogonalize(z)
    assert (got[0] == 0).all()
    close(got[1], iterate(z[1]), HALF["bf16"])
    for size in (1e-30, 1e30, 1e-42):                          # the norm's square would leave binary32's range
        x = matrix(65, 70, "plain", 4) * size
        close(zpq.orthogonalize(x), iterate(x), HALF["bf16"])
    for bad in (float("nan"), float("inf")):
        x = matrix(70, 90, "plain", 5, 3)
        x[1, 3, 7] = bad
        got = zpq.orthogonalize(x)
        assert got[1].isnan().all()
        close(got[0], iterate(x[0]), HALF["bf16"])
        close(got[2], iterate(x[2]), HALF["bf16"])
    assert zpq.orthogonalize(torch.zeros(0, 5, device="cuda")).shape == (0, 5)
    assert zpq.orthogonalize(torch.zeros(2, 5, 0, device="cuda")).shape == (2, 5, 0)
    assert zpq.orthogonalize(torch.zeros(0, 5, 6, device="cuda")).shape == (0, 5, 6)


def test_orthogonalize_repeats_bit_for_bit():
    x = matrix(300, 1000, "strong", 6)
    first = zpq.orthogonalize(x)
    for _ in range(4):
        assert torch.equal(zpq.orthogonalize(x), first)


# ------------------------------------------------------------------------------------------- Muon
LAYER = [(96, 32), (32, 32), (128, 32), (32, 128), (1, 50), (77, 3), (200, 333), (64, 192), (200, 48)]


def make(shapes, p="f32", g="bf16", copy=None, seed=0, **options):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    t = dict(p=[(rand(s) * 0.02).to(DT[p]) for s in shapes], g=[(rand(s) * 1e-3).to(DT[g]) for s in shapes],
             m=[rand(s) * 3e-3 for s in shapes], copy=None if copy is None else [torch.zeros(s, dtype=DT[copy], device="cuda") for s in shapes])
    before = {k: None if v is None else [x.double().clone() for x in v] for k, v in t.items()}
    opt = zpq.Muon(t["p"], t["g"], copies=t["copy"], momenta=t["m"], **options)
    return opt, t, before


def expected(before, i, lr, momentum, nesterov, decay, scale, c):
    g = before["g"][i] * c
    m = momentum * before["m"][i] + g
    o = iterate(g + momentum * m if nesterov else m)
    return m, before["p"][i] * (1 - lr * decay), -lr * scale * o


def check(t, before, i, m, kept, update, half_p):
    # the momentum: two products, a sum, rounded constants
    assert ((t["m"][i].double() - m).abs() <= 4 * 2.0 ** -24 * (before["m"][i].abs() + before["g"][i].abs())).all()
    got, size = t["p"][i].double(), update.square().mean().sqrt()
    slack = 3 * 2.0 ** -24 * before["p"][i].abs() + half_p * (kept + update).abs()
    d = (got - kept - update).abs()
    assert (d <= 8 * 2.0 ** -8 * size + slack).all()
    if t["copy"] is not None:
        assert torch.equal(t["copy"][i], t["p"][i].to(t["copy"][i].dtype))


@pytest.mark.parametrize("p,g,copy", [("f32", "bf16", "bf16"), ("f32", "f32", None), ("f32", "f16", "f16"), ("bf16", "bf16", None), ("f16", "f32", None)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_step(p, g, copy, nesterov):
    decay = [0.1 * (i % 3) for i in range(len(LAYER))]
    opt, t, before = make(LAYER, p, g, copy, lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=decay)
    opt.step(lr=0.03, grad_scale=0.5)
    for i, (r, c) in enumerate(LAYER):
        want = expected(before, i, 0.03, 0.9, nesterov, decay[i], 0.2 * max(r, c) ** 0.5, 0.5)
        check(t, before, i, *want, {"f32": 2.0 ** -24, **HALF}[p])


def test_muon_clips_and_stops():
    opt, t, before = make(LAYER, copy="bf16", lr=0.02)
    total = opt.grad_sumsq()
    assert abs(total.item() / sum(x.square().sum().item() for x in before["g"]) - 1) < 1e-12
    opt.step(sumsq=total, max_norm=1e-2)
    c = 1e-2 / (total.item() ** 0.5 + 1e-6)
    for i, (rows, cols) in enumerate(LAYER):
        check(t, before, i, *expected(before, i, 0.02, 0.95, True, 0.0, 0.2 * max(rows, cols) ** 0.5, c), 2.0 ** -24)
    after = [x.clone() for k in ("p", "m", "copy") for x in t[k]]
    for bad in (float("inf"), float("nan")):
        opt.step(sumsq=torch.full((1,), bad, dtype=torch.float64, device="cuda"), max_norm=1.0)
        assert all(torch.equal(a, b) for a, b in zip(after, (x for k in ("p", "m", "copy") for x in t[k])))


def test_muon_many_and_empty():
    """More matrices than one launch describes, empty ones among them; given scales."""
    shapes = [(s, s + 7) if s % 5 else (s, 0) for s in range(45)]
    opt, t, before = make(shapes, lr=0.1, scale=[0.5 + i for i in range(45)])
    opt.step()
    for i, s in enumerate(shapes):
        if s[0] * s[1]:
            check(t, before, i, *expected(before, i, 0.1, 0.95, True, 0.0, 0.5 + i, 1.0), 2.0 ** -24)


def test_muon_more_than_it_works_on_at_a_time():
    """Three matrices of 36 M elements go one after the other through the same memory."""
    shapes = [(6000, 6010), (30, 40), (6010, 6000), (6000, 6000), (50, 20)]
    opt, t, before = make(shapes, lr=0.02, steps=1)
    assert opt._memory.numel() < 20 * 6010 * 6010
    opt.step()
    for i, s in enumerate(shapes):
        g = before["g"][i]
        m = 0.95 * before["m"][i] + g
        want = -0.02 * 0.2 * max(s) ** 0.5 * iterate(g + 0.95 * m, (TRIPLE,))
        check(t, before, i, m, before["p"][i], want, 2.0 ** -24)


def test_muon_set_grads_and_zeros():
    opt, t, before = make(LAYER, lr=0.02)
    opt.set_grads([torch.zeros_like(g) for g in t["g"]])
    for m in t["m"]:
        m.zero_()
    opt.step()
    assert all(torch.equal(a.double(), b) for a, b in zip(t["p"], before["p"]))     # no update, no decay
    with pytest.raises(ValueError, match="grads: need torch.bfloat16"):
        opt.set_grads([g.float() for g in t["g"]])
    with pytest.raises(ValueError, match="overlap"):
        opt.set_grads([m.view(torch.bfloat16).view(-1)[:m.numel()].view(m.shape) for m in t["m"]])


def test_captured_steps():
    """A graph of the norm and the step, replayed with new gradients and eager work between, equals eager steps."""
    opt, t, _ = make(LAYER, copy="bf16", lr=0.02, weight_decay=0.1)
    twin, u, _ = make(LAYER, copy="bf16", lr=0.02, weight_decay=0.1)
    x = matrix(70, 150, "strong", 9)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        opt.step(sumsq=opt.grad_sumsq(), max_norm=1.0)
        zpq.orthogonalize(x)
    torch.cuda.synchronize()
    twin.step(sumsq=twin.grad_sumsq(), max_norm=1.0)
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.grad_sumsq(out=total)
        opt.step(sumsq=total, max_norm=1.0)
        o = zpq.orthogonalize(x)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for k in range(5):
        for a, b in zip(t["g"], u["g"]):
            a.copy_(torch.randn(a.shape, generator=gen, device="cuda") * 1e-3)
            b.copy_(a)
        x.copy_(matrix(70, 150, "strong", 20 + k))
        graph.replay()
        twin.step(sumsq=twin.grad_sumsq(), max_norm=1.0)
        torch.cuda.synchronize()
        for name in ("p", "m", "copy"):
            assert all(torch.equal(a, b) for a, b in zip(t[name], u[name]))
        assert torch.equal(o, zpq.orthogonalize(x))
