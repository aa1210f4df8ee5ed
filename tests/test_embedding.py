"""The embedding lookup and its gradient on the GPU, against 64-bit
definitions (step_ref)."""
import numpy as np
import pytest

import block_quantized_communication_amd as zpq
import step_ref as ref

pytestmark = pytest.mark.gpu
TYPES = ["f32", "f16", "bf16"]


def tdt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def host(t):
    return t.detach().double().cpu().numpy()


def rounded(x, dt, roundings):
    """Tolerance of a value computed in binary32 with that many roundings and
    rounded once into dt."""
    return ref.U * roundings * np.abs(x) + (0 if dt == "f32" else ref.HALF[dt] * np.abs(x) * (1 + 1e-6)) + ref.TINY[dt]


def draw_ids(n, rows, seed, first=0, bad=True, width="i64"):
    """Frequent and rare rows, and ids on both sides of the table."""
    import torch
    rng = np.random.default_rng(seed)
    ids = np.floor(np.exp(rng.uniform(0, np.log(rows + 1), n)) - 1).astype(np.int64).clip(0, rows - 1) + first
    if bad and n > 3:
        ids[rng.integers(0, n, max(1, n // 10))] = first - 1
        ids[rng.integers(0, n, max(1, n // 10))] = first + rows
        ids[0] = -(1 << 31) if width == "i32" else -(1 << 62)
    t = torch.from_numpy(ids.astype(np.int32 if width == "i32" else np.int64)).cuda()
    return ids, t


@pytest.mark.parametrize("table", TYPES)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("tokens,rows,dim", [(1, 1, 1), (5, 3, 7), (300, 50, 8), (64, 17, 13), (33, 100, 256),
                                             (1000, 999, 129)])
def test_lookup(table, out, tokens, rows, dim):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(dim)
    w = torch.randn(rows, dim, generator=gen, device="cuda").to(tdt(table))
    ids, t = draw_ids(tokens, rows, dim)
    y = zpq.embedding(t, w, scale=1.7, out_dtype=tdt(out))
    want = ref.lookup64(ids, host(w), float(np.float32(1.7)))
    assert y.shape == (tokens, dim) and y.dtype == tdt(out)
    assert np.all(np.abs(host(y) - want) <= rounded(want, out, 1))


@pytest.mark.parametrize("width", ["i32", "i64"])
@pytest.mark.parametrize("first", [0, 1000, -5])
def test_lookup_of_a_shard(width, first):
    """Rows [first, first + rows) of a vocabulary: the others give zeros."""
    import torch
    w = torch.arange(60 * 24, device="cuda", dtype=torch.float32).view(60, 24) + 1
    ids, t = draw_ids(400, 60, 4, first=first, width=width)
    y = zpq.embedding(t, w, first=first)
    assert np.array_equal(host(y), ref.lookup64(ids, host(w), 1.0, first))


@pytest.mark.parametrize("dim", [5, 16, 21])
def test_lookup_strides_shapes_and_out(dim):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(40, dim + 9, generator=gen, device="cuda").half()[:, 3:3 + dim]      # rows apart, misaligned
    ids, t = draw_ids(60, 40, 2)
    want = ref.lookup64(ids, host(w), 1.0)
    assert np.array_equal(host(zpq.embedding(t.view(3, 4, 5), w)).reshape(60, dim), want)
    big = torch.full((60, dim + 5), 7.0, device="cuda")
    zpq.embedding(t, w, out=big[:, 2:2 + dim])
    assert np.array_equal(host(big[:, 2:2 + dim]), want)
    assert bool((big[:, :2] == 7).all()) and bool((big[:, 2 + dim:] == 7).all())
    with pytest.raises(ValueError):
        zpq.embedding(t, w.t())
    with pytest.raises(ValueError):
        zpq.embedding(t.float(), w)
    with pytest.raises(ValueError):
        zpq.embedding(t, w, out=torch.empty(59, dim, device="cuda"))
    assert zpq.embedding(t[:0], w).shape == (0, dim)


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("block", [32, 64, 128, 256, 512])
@pytest.mark.parametrize("rows,dim", [(64, 512), (100, 24), (33, 33), (7, 3), (50, 1001)])
def test_lookup_int8(out, block, rows, dim):
    """From qwZ's codes and scales, rows that are no whole blocks among them."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(block + dim)
    n = -(-rows * dim // block) * block
    x = torch.randn(n, generator=gen, device="cuda") * 0.02
    codes, scales = zpq.quant_i8(x, block)
    ids, t = draw_ids(200, rows, dim)
    y = zpq.embedding_i8(t, codes, scales, rows, dim, block=block, scale=3.0, out_dtype=tdt(out))
    w = codes.cpu().numpy().astype(np.float64) * np.repeat(host(scales), block)
    want = ref.lookup64(ids, w[:rows * dim].reshape(rows, dim), 3.0)
    assert np.all(np.abs(host(y) - want) <= rounded(want, out, 2))
    dense = zpq.dequant_i8(codes, scales, block, torch.float32)[:rows * dim].view(rows, dim)
    assert torch.equal(zpq.embedding(t, dense, scale=3.0, out_dtype=tdt(out)), y)


def test_lookup_past_32_bits():
    """Table and output offsets beyond 2^32 elements, more lanes than one launch
    takes."""
    import torch
    rows, dim, n = (1 << 20) + 8, 4096, (1 << 21) + 3
    codes = torch.zeros(rows * dim, dtype=torch.int8, device="cuda")
    scales = torch.full((rows * dim // 256,), 0.5, device="cuda")
    codes.view(rows, dim)[-1] = 3
    codes.view(rows, dim)[1] = 5
    t = torch.full((n,), rows - 1, device="cuda")
    t[:2] = 1
    t[-2] = 1
    y = zpq.embedding_i8(t, codes, scales, rows, dim, scale=2.0)
    assert bool((y[:2] == 5).all()) and bool((y[-2] == 5).all()) and bool((y[-1] == 3).all())
    assert int((y[:, 0] != 3).sum()) == 3 and int((y[:, -1] != 3).sum()) == 3


def test_lookup_without_rows():
    import torch
    t = torch.arange(5, device="cuda")
    y = zpq.embedding(t, torch.empty(0, 24, device="cuda").half())
    assert y.shape == (5, 24) and not bool(y.any())
    y = zpq.embedding_i8(t, torch.empty(0, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"), 0, 24)
    assert y.shape == (5, 24) and not bool(y.any())


def terms_off(n):
    """Roundings in a row's sum of n terms: one an addition, and a term passes
    through at most 63 additions in each group level and 2 * 63 a level in its
    row (4 levels are more than any test here has)."""
    return np.minimum(n, 64 * 12)


def check_grad(got, base, ids, dy, rows, scale, out, **kw):
    g, mag, n = ref.grad64(ids, dy, rows, float(np.float32(scale)), **kw)
    want = g + base
    tol = ref.U * ((terms_off(n)[:, None] + 2) * mag + np.abs(want) + np.abs(base)) + \
        (0 if out == "f32" else ref.HALF[out] * (np.abs(want) + ref.U * 800 * mag)) + ref.TINY[out]
    d = np.abs(got - want)
    assert np.all(d <= tol), (np.max(d - tol), np.argwhere(d > tol)[:3])
    assert np.array_equal(got[n == 0], base[n == 0] if isinstance(base, np.ndarray) else np.zeros_like(got[n == 0]))


@pytest.mark.parametrize("dy", TYPES)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,rows,dim", [(0, 5, 8), (1, 1, 1), (6, 4, 7), (200, 30, 12), (700, 1000, 33),
                                             (3000, 257, 64)])
def test_grad(dy, out, accumulate, tokens, rows, dim):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    y = torch.randn(tokens, dim, generator=gen, device="cuda").to(tdt(dy))
    ids, t = draw_ids(tokens, rows, tokens)
    if accumulate:
        g = torch.randn(rows, dim, generator=gen, device="cuda").to(tdt(out))
        base = host(g)
        assert zpq.embedding_grad(t, y, rows, scale=0.7, out=g, accumulate=True) is g
    else:
        g = zpq.embedding_grad(t, y, rows, scale=0.7, out_dtype=tdt(out))
        base = np.zeros((rows, dim))
    check_grad(host(g), base, ids, host(y), rows, 0.7, out)


@pytest.mark.parametrize("tokens", [255, 256, 257, 1024, 1025, 4095, 4096, 4097, 5119, 5121, 16384, 16385, 20481, 24576,
                                    24577, 32768, 32769, 140000])
@pytest.mark.parametrize("kind", ["frequent", "one", "spread"])
def test_grad_sizes_of_the_sort(tokens, kind):
    """Every number of runs and group levels: exact sums of small integers."""
    import torch
    rows, dim = 5000, 16
    rng = np.random.default_rng(tokens)
    ids = {"frequent": lambda: draw_ids(tokens, rows, 3, bad=True)[0], "one": lambda: np.full(tokens, 4321),
           "spread": lambda: rng.integers(-1, rows + 1, tokens)}[kind]()
    y = rng.integers(-8, 9, (tokens, dim))                 # sums of less than 2^24: exact
    g = zpq.embedding_grad(torch.from_numpy(ids).cuda(), torch.from_numpy(y.astype(np.float32)).cuda().bfloat16(), rows,
                           out_dtype=torch.float32)
    want, _, _ = ref.grad64(ids, y.astype(np.float64), rows, 1.0)
    assert np.array_equal(host(g), want)


def test_grad_order_is_fixed_by_the_ids():
    import torch
    ids, t = draw_ids(50000, 300, 5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    y = torch.randn(50000, 40, generator=gen, device="cuda")
    a = zpq.embedding_grad(t, y, 300)
    for _ in range(3):
        assert torch.equal(a, zpq.embedding_grad(t, y, 300))
    assert torch.equal(a, zpq.embedding_grad(t.int() if abs(ids).max() < 2 ** 31 else t, y, 300))
    check_grad(host(a), np.zeros((300, 40)), ids, host(y), 300, 1.0, "f32")


@pytest.mark.parametrize("width", ["i32", "i64"])
def test_grad_of_a_shard_with_padding(width):
    import torch
    ids, t = draw_ids(900, 70, 8, first=200, width=width)
    gen = torch.Generator(device="cuda").manual_seed(6)
    y = torch.randn(900, 24, generator=gen, device="cuda").half()
    g = zpq.embedding_grad(t, y, 70, first=200, padding=200, out_dtype=torch.float32)
    check_grad(host(g), np.zeros((70, 24)), ids, host(y), 70, 1.0, "f32", first=200, padding=200)
    assert not bool(g[0].any())


@pytest.mark.parametrize("dim", [5, 20])
def test_grad_strides(dim):
    """Rows of dy and of the gradient apart and misaligned; what lies between
    stays."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(9)
    y = torch.randn(500, dim + 6, generator=gen, device="cuda").half()[:, 1:1 + dim]
    ids, t = draw_ids(500, 64, 9)
    for acc in (False, True):
        big = torch.full((64, dim + 7), 2.0, device="cuda").bfloat16()
        base = np.full((64, dim), 2.0 if acc else 0.0)
        zpq.embedding_grad(t, y, 64, out=big[:, 3:3 + dim], accumulate=acc)
        check_grad(host(big[:, 3:3 + dim]), base, ids, host(y), 64, 1.0, "bf16")
        assert bool((big[:, :3] == 2).all()) and bool((big[:, 3 + dim:] == 2).all())


def test_grad_is_the_gradient_of_the_lookup():
    """Against differences: <dy, lookup(W + h V) - lookup(W)> = h <grad, V>,
    exact for a linear map up to the roundings of the sums."""
    import torch
    rng = np.random.default_rng(11)
    rows, dim, tokens = 37, 48, 600
    ids, t = draw_ids(tokens, rows, 12)
    w = torch.from_numpy(rng.integers(-64, 65, (rows, dim)).astype(np.float32)).cuda()
    v = torch.from_numpy(rng.integers(-64, 65, (rows, dim)).astype(np.float32)).cuda()
    y = torch.from_numpy(rng.integers(-64, 65, (tokens, dim)).astype(np.float32)).cuda()
    change = zpq.embedding(t, w + v, scale=0.5) - zpq.embedding(t, w, scale=0.5)     # exact: small integers / 2
    g = zpq.embedding_grad(t, y, rows, scale=0.5)
    assert (y.double() * change.double()).sum().item() == (g.double() * v.double()).sum().item()


def test_grad_infinities_stay_in_their_rows():
    import torch
    ids = torch.tensor([0, 1, 1, 3, -1], device="cuda")
    y = torch.ones(5, 16, device="cuda")
    y[1, 2], y[3, 5], y[4, 7] = float("inf"), float("nan"), float("nan")
    g = host(zpq.embedding_grad(ids, y, 4))
    want = np.zeros((4, 16))
    want[0], want[1], want[3] = 1, 2, 1
    want[1, 2], want[3, 5] = np.inf, np.nan
    assert np.array_equal(g, want, equal_nan=True)


def test_grad_refusals():
    import torch
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    y = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        zpq.embedding_grad(t, y[:3], 10)
    with pytest.raises(ValueError):
        zpq.embedding_grad(t, y, 10, accumulate=True)
    with pytest.raises(ValueError):
        zpq.embedding_grad(t, y, 10, out=torch.zeros(9, 8, device="cuda"))
    with pytest.raises(ValueError):
        zpq.embedding_grad(t, y.double(), 10)
    with pytest.raises(ValueError):
        zpq.embedding_grad(t, y.t().contiguous().t(), 10)
    with pytest.raises(zpq.ZpqError):
        zpq.embedding_grad(t, y, 4, out=y, accumulate=True)              # in place


def test_other_stream_and_graph():
    import torch
    rows, dim, n = 500, 96, 3000
    ids, t = draw_ids(n, rows, 13)
    gen = torch.Generator(device="cuda").manual_seed(14)
    w = torch.randn(rows, dim, generator=gen, device="cuda").half()
    g = torch.zeros(rows, dim, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = zpq.embedding(t, w, scale=2.0, stream=side)
    zpq.embedding_grad(t, y, rows, out=g, stream=side)
    side.synchronize()
    want = zpq.embedding(t, w, scale=2.0)
    assert torch.equal(y, want)
    assert torch.equal(g, zpq.embedding_grad(t, want, rows, out_dtype=torch.float32))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = zpq.embedding(t, w, scale=2.0)
        zpq.embedding_grad(t, y, rows, out=g)
    for rep in range(4):
        print(f"graph replay {rep}", flush=True)
        ids, new = draw_ids(n, rows, 20 + rep)
        t.copy_(new)
        w.copy_(torch.randn(rows, dim, generator=gen, device="cuda").half())
        want = zpq.embedding(t, w, scale=2.0)
        grad = zpq.embedding_grad(t, want, rows, out_dtype=torch.float32)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(g, grad), rep


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,rows,dim", [(53280, 4, 24), (8192, 2048, 12), (4096, 4096, 12), (4096, 4097, 12), (8193, 3, 520),
                                             (511, 70, 9), (512, 70, 9), (20000, 90000, 132), (300000, 5, 7),
                                             (3000, 40, 12000), (2500, 200000, 3), (9000, 300000, 6)])
def test_grad_sizes_of_the_sums(tokens, rows, dim, accumulate):
    """Both sides of the rules on group sizes and levels, on where the rows' places
    are found and on launches over tokens: exact sums of small integers."""
    import torch
    rng = np.random.default_rng(tokens + rows)
    ids, t = draw_ids(tokens, rows, rows)
    y = rng.integers(-2, 3, (tokens, dim))
    g = torch.full((rows, dim), 3.0, device="cuda")
    zpq.embedding_grad(t, torch.from_numpy(y.astype(np.float32)).cuda().half(), rows, scale=2.0, out=g,
                       accumulate=accumulate)
    want, _, _ = ref.grad64(ids, y.astype(np.float64), rows, 2.0)
    assert np.array_equal(host(g), want + (3.0 if accumulate else 0.0))


def test_grad_past_32_bits():
    """dy and the gradient beyond 2^32 elements, more waves than one launch takes."""
    import torch
    rows = tokens = (1 << 21) + 9
    dim = 4100
    y = torch.zeros(tokens, dim, dtype=torch.bfloat16, device="cuda")
    y[-1], y[-2], y[3] = 3.0, 5.0, 7.0
    t = torch.full((tokens,), -1, device="cuda")
    t[-1] = t[3] = rows - 1
    t[-2] = rows - 2
    g = zpq.embedding_grad(t, y, rows)
    assert bool((g[-1] == 10).all()) and bool((g[-2] == 5).all()) and not bool(g[:-2].any())
    zpq.embedding_grad(t, y, rows, out=g, accumulate=True)
    assert bool((g[-1] == 20).all()) and bool((g[-2] == 10).all()) and not bool(g[5:9].any())


def test_grad_of_more_lanes_than_one_launch():
    """Short rows, dealt out lane by lane."""
    import torch
    rows, dim = (1 << 26) + 5, 136
    t = torch.tensor([rows - 1, 0, rows - 1, 1 << 25, rows - 2], device="cuda")
    y = torch.arange(1, 6, device="cuda").bfloat16()[:, None].expand(5, dim).contiguous()
    g = zpq.embedding_grad(t, y, rows)
    assert bool((g[-1] == 4).all()) and bool((g[0] == 2).all()) and bool((g[1 << 25] == 4).all())
    assert bool((g[-2] == 5).all()) and not bool(g[1:1 << 25].any()) and not bool(g[(1 << 25) + 1:-2].any())


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens", [1, 5, 64, 65, 255, 257, 600])
@pytest.mark.parametrize("rows", [(1 << 16) - 1, 1 << 16, (1 << 16) + 1, 1 << 20])
def test_grad_of_few_tokens_into_many_rows(tokens, rows, accumulate):
    """Both sides of the rule on where the rows' places are found that goes by the
    rows alone: exact sums of small integers, first and last rows among them."""
    import torch
    rng = np.random.default_rng(tokens)
    ids = rng.choice([0, 1, rows // 2, rows - 2, rows - 1, rows, -1, 63, 64, 65], tokens)
    y = rng.integers(-2, 3, (tokens, 8))
    g = torch.full((rows, 8), 3.0, device="cuda")
    zpq.embedding_grad(torch.from_numpy(ids).cuda(), torch.from_numpy(y.astype(np.float32)).cuda(), rows, scale=2.0,
                       out=g, accumulate=accumulate)
    want, _, _ = ref.grad64(ids, y.astype(np.float64), rows, 2.0)
    assert np.array_equal(host(g), want + (3.0 if accumulate else 0.0))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tokens,rows", [(900, 300), (3000, 300), (3000, 90000), (20000, 300), (24576, 70000), (50000, 300),
                                         (140000, 70000)])
def test_grad_with_ids_of_4_bytes(tokens, rows, accumulate):
    """Every way of sorting, from both widths of the same ids (negative and too large
    ones among them): the same bits, and the exact sums of small integers."""
    import torch
    ids, t = draw_ids(tokens, rows, 5, width="i32")
    assert t.dtype == torch.int32 and ids.min() == -(1 << 31) and ids.max() >= rows
    y = np.random.default_rng(6).integers(-8, 9, (tokens, 12))
    dy = torch.from_numpy(y.astype(np.float32)).cuda()
    g = [torch.full((rows, 12), 5.0, device="cuda") for _ in range(2)]
    zpq.embedding_grad(t, dy, rows, padding=7, out=g[0], accumulate=accumulate)
    zpq.embedding_grad(t.long(), dy, rows, padding=7, out=g[1], accumulate=accumulate)
    assert torch.equal(g[0], g[1])
    want, _, _ = ref.grad64(ids, y.astype(np.float64), rows, 1.0, padding=7)
    assert np.array_equal(host(g[0]), want + (5.0 if accumulate else 0.0))
    z = torch.randn(tokens, 40, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    assert torch.equal(zpq.embedding_grad(t, z, rows), zpq.embedding_grad(t.long(), z, rows))
