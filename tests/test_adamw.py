"""The optimizer step, the gradient norm and the 8-bit states on the GPU,
against step_ref's definitions.  8-bit codes and exponents must be equal;
floats within the roundings that step_ref.adamw64 counts."""
import math

import numpy as np
import pytest

import block_quantized_communication_amd as zpq
import step_ref as ref

pytestmark = pytest.mark.gpu
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8)


def tdt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def host(t):
    return t.detach().double().cpu().numpy()


def make(sizes, p="f32", g="bf16", copy="bf16", bits=32, seed=0, offset=0, clean=True):
    """Tensors of the given sizes; offset > 0: views that start that many
    elements into an allocation (misaligned)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(n, scale, dt):
        x = torch.randn(n + offset, generator=gen, device="cuda") * scale
        return x.to(dt)[offset:]

    d = dict(p=[], g=[], m=[], v=[], copy=[] if copy else None)
    for i, n in enumerate(sizes):
        s = 10.0 ** (-1 - i % 4)
        d["p"].append(rnd(n, 0.05, tdt(p)))
        d["g"].append(rnd(n, s, tdt(g)))
        m, v = rnd(n, s * 0.3, torch.float32), (rnd(n, s, torch.float32) ** 2)
        if bits == 8:
            at = lambda pair: tuple(torch.cat([torch.zeros(offset, dtype=torch.uint8, device="cuda"), x])[offset:]  # noqa: E731
                                    for x in pair)
            d["m"].append(at(zpq.state8_pack(m.contiguous(), 1)))
            d["v"].append(at(zpq.state8_pack(v.contiguous(), 2)))
        else:
            d["m"].append(m)
            d["v"].append(v)
        if copy:
            d["copy"].append(torch.zeros(n + offset, dtype=tdt(copy), device="cuda")[offset:])
    return d


def state_of(x, moment):
    """float64 values of a state tensor or pair."""
    if isinstance(x, tuple):
        return ref.decode8(x[0].cpu().numpy(), x[1].cpu().numpy(), moment)
    return host(x)


def run(d, bits, step=3, seed=7, decay=0.1, max_norm=None, grad_scale=1.0, use_sum=True, stream=None):
    opt = zpq.AdamW(d["p"], d["g"], copies=d["copy"], state_bits=bits, exp_avg=d["m"], exp_avg_sq=d["v"], seed=seed,
                    weight_decay=decay, stream=stream, **HYPER)
    total = opt.grad_sumsq(stream=stream) if use_sum else None
    opt.step(step, sumsq=total, max_norm=max_norm, grad_scale=grad_scale, stream=stream)
    return opt, total


def check(d0, d, bits, p, copy, total, step=3, seed=7, decay=0.1, max_norm=None, grad_scale=1.0):
    """d: after the step; d0: (p, g, m, v) float64 before it, per tensor."""
    want = sum(float((g ** 2).sum()) for _, g, _, _ in d0)
    if total is not None:
        # binary64 sums of exact squares: at most one rounding an addition
        assert abs(total.item() - want) <= 2.0 ** -52 * want * (4 + math.log2(2 + sum(x[0].size for x in d0))) * 64
    c = ref.clip_factor(None if total is None else total.item(), grad_scale, max_norm or math.inf)
    base = 0
    decay = decay if isinstance(decay, list) else [decay] * len(d0)
    for i, (p0, g0, m0, v0) in enumerate(d0):
        n = p0.size
        p1, m1, v1, tp, tm, tv = ref.adamw64(p0, g0, m0, v0, c, HYPER["lr"], HYPER["betas"], HYPER["eps"], decay[i], step)
        got = host(d["p"][i])
        tol = tp + (0 if p == "f32" else ref.HALF[p] * (np.abs(p1) + tp) + ref.TINY[p])
        assert np.all(np.abs(got - p1) <= tol), (i, n, np.max(np.abs(got - p1) - tol))
        if copy:
            assert np.array_equal(host(d["copy"][i]), host(d["p"][i].to(tdt(copy)))), (i, n)
        if bits == 32:
            assert np.all(np.abs(host(d["m"][i]) - m1) <= tm), (i, n)
            assert np.all(np.abs(host(d["v"][i]) - v1) <= tv), (i, n)
        else:
            ms, vs = ref.adamw32_moments(g0, m0, v0, c, HYPER["betas"])
            r = ref.random32(base, n, seed, step)
            for x, moment, rnd, got in ((ms, 1, r & 0xFFFF, d["m"][i]), (vs, 2, r >> 16, d["v"][i])):
                codes, exps = ref.encode8(x, moment, rnd)
                assert np.array_equal(got[1].cpu().numpy(), exps), (i, n, moment)
                assert np.array_equal(got[0].cpu().numpy(), codes), (i, n, moment)
        base += ref.padded(n)


def before(d):
    return [(host(p), host(g), state_of(m, 1), state_of(v, 2)) for p, g, m, v in zip(d["p"], d["g"], d["m"], d["v"])]


SIZES = {"one": [1], "short": [7, 8, 9, 0, 255, 256, 257], "tiles": [2047, 2048, 2049, 4096, 0, 5],
         "many": [1 + (i * 37) % 300 for i in range(70)], "very many": [1 + i % 13 for i in range(4200)],
         "large": [3 * 2048 * 100 + 11]}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_sizes(sizes, bits):
    d = make(SIZES[sizes], bits=bits)
    d0 = before(d)
    _, total = run(d, bits, max_norm=1.0)
    check(d0, d, bits, "f32", "bf16", total, max_norm=1.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("p,copy", [("f32", None), ("f32", "f16"), ("f32", "bf16"), ("f16", None), ("bf16", None)])
@pytest.mark.parametrize("offset", [0, 1])
def test_types_and_alignment(p, g, copy, bits, offset):
    d = make([5000, 3, 2048], p=p, g=g, copy=copy, bits=bits, offset=offset, seed=3)
    d0 = before(d)
    _, total = run(d, bits, decay=[0.1, 0.0, 0.5])
    check(d0, d, bits, p, copy, total, decay=[0.1, 0.0, 0.5])


@pytest.mark.parametrize("bits", [32, 8])
def test_scale_without_norm_and_first_step(bits):
    """No norm given, gradients scaled, states made by the optimizer."""
    d = make([1000, 300], bits=bits, g="f32")
    opt = zpq.AdamW(d["p"], d["g"], copies=d["copy"], state_bits=bits, seed=1, weight_decay=0.0, **HYPER)
    d["m"], d["v"] = opt.exp_avg, opt.exp_avg_sq
    d0 = before(d)
    assert all(not m.any() and not v.any() for _, _, m, v in d0)
    opt.step(1, grad_scale=0.125)
    check(d0, d, bits, "f32", "bf16", None, step=1, seed=1, decay=0.0, grad_scale=0.125)


def test_many_steps_follow_64_bits():
    """200 steps on a quadratic, weights 8 and 32 bits, against float64 steps:
    32-bit states stay with it, 8-bit states end as near the minimum."""
    import torch
    n = 4096
    gen = torch.Generator(device="cuda").manual_seed(5)
    target = torch.randn(n, generator=gen, device="cuda")
    scale = 10.0 ** (torch.rand(n, generator=gen, device="cuda") * 2 - 1)
    end = {}
    for bits in (32, 8):
        p = torch.zeros(n, device="cuda")
        g = torch.zeros(n, device="cuda")
        opt = zpq.AdamW([p], [g], lr=0.02, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0, state_bits=bits, seed=9)
        for t in range(1, 201):
            g.copy_((p - target) * scale)
            opt.step(t)
        end[bits] = p.cpu().numpy()
    p, m, v = np.zeros(n), np.zeros(n), np.zeros(n)
    tg, sc = host(target), host(scale)
    for t in range(1, 201):
        p, m, v, *_ = ref.adamw64(p, (p - tg) * sc, m, v, 1.0, 0.02, (0.9, 0.99), 1e-8, 0.0, t)
    # 200 steps of at most lr each, every one within 2^-19 of its size (the counted
    # roundings, about 30 half-steps), amplified by no more than the steps there are
    assert np.max(np.abs(end[32] - p)) < 200 * 0.02 * 2.0 ** -19 * 20
    away = lambda x: float(np.sqrt(np.mean((x - tg) ** 2)))  # noqa: E731
    assert away(end[8]) < 1.1 * away(p) + 0.02           # within one step's length


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_changes_nothing(bits, bad):
    d = make([3000, 10], bits=bits)
    d["g"][1][4] = bad
    flat = lambda xs: [y.clone() for x in xs for y in (x if isinstance(x, tuple) else (x,))]  # noqa: E731
    old = flat(d["p"] + d["copy"] + d["m"] + d["v"])
    _, total = run(d, bits, max_norm=1.0)
    assert not math.isfinite(total.item())
    for a, b in zip(old, flat(d["p"] + d["copy"] + d["m"] + d["v"])):
        assert np.array_equal(a.view(a.dtype).cpu().float().numpy(), b.cpu().float().numpy())


def test_infinite_gradient_without_a_norm_marks_its_block():
    """8-bit states: the block of the bad element becomes infinite as a whole,
    the others are as ever."""
    d = make([256 * 4], bits=8, g="f32")
    d["g"][0][300] = float("inf")
    d0 = before(d)
    run(d, 8, use_sum=False)
    (mc, me), (vc, ve) = d["m"][0], d["v"][0]
    assert me.cpu()[1] == 255 and ve.cpu()[1] == 255
    assert bool((mc[256:512] == 127).all()) and bool((vc[256:512] == 255).all())
    assert np.all(np.isinf(ref.decode8(vc.cpu().numpy(), ve.cpu().numpy(), 2)[256:512]))
    p0, g0, m0, v0 = (x[512:] for x in d0[0])
    p1, _, _, tp, _, _ = ref.adamw64(p0, g0, m0, v0, 1.0, HYPER["lr"], HYPER["betas"], HYPER["eps"], 0.1, 3)
    assert np.all(np.abs(host(d["p"][0])[512:] - p1) <= tp)


def test_extreme_magnitudes_of_8_bit_states():
    """Gradients from subnormal squares to the top of the range, zero blocks,
    blocks of one value: codes as defined."""
    import torch
    rows = []
    gen = np.random.default_rng(3)
    for s in (1e-30, 1e-22, 1e-19, 1e-10, 1.0, 1e10, 1e18):
        rows.append(gen.standard_normal(256) * s)
    rows.append(np.zeros(256))
    rows.append(np.full(256, 1.875))
    rows.append(np.full(256, 1.9))
    rows.append(np.where(np.arange(256) == 9, 1e3, 1e-9))
    x = np.concatenate(rows).astype(np.float32)
    g = torch.from_numpy(x).cuda()
    n = x.size
    d = dict(p=[torch.zeros(n, device="cuda")], g=[g], copy=None)
    opt = zpq.AdamW(d["p"], d["g"], state_bits=8, seed=7, weight_decay=0.1, **HYPER)
    d["m"], d["v"] = opt.exp_avg, opt.exp_avg_sq
    d0 = before(d)
    opt.step(3)
    check(d0, d, 8, "f32", None, None)
    d0 = before(d)                                   # and on from those states
    opt.step(4)
    check(d0, d, 8, "f32", None, None, step=4)


@pytest.mark.parametrize("moment", [1, 2])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 256, 257, 5000])
def test_pack_and_unpack(moment, dt, n):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = (torch.randn(n, generator=gen, device="cuda") * 0.01).to(tdt(dt))
    if moment == 2:
        x = x.abs()
    codes, exps = zpq.state8_pack(x, moment)
    want_c, want_e = ref.encode8(x.float().cpu().numpy(), moment)
    assert np.array_equal(exps.cpu().numpy(), want_e) and np.array_equal(codes.cpu().numpy(), want_c)
    values = ref.decode8(want_c, want_e, moment)
    got = zpq.state8_unpack(codes, exps, moment, dtype=tdt(dt))
    want = torch.from_numpy(values).to(tdt(dt)).double().numpy()
    assert np.array_equal(host(got), want)


@pytest.mark.parametrize("moment", [1, 2])
def test_unpack_every_code_and_exponent(moment):
    import torch
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(255).cuda()
    exps = torch.arange(1, 256, dtype=torch.int32).to(torch.uint8).cuda()
    got = zpq.state8_unpack(codes, exps, moment).cpu().numpy()
    with np.errstate(over="ignore"):
        want = ref.decode8(codes.cpu().numpy(), exps.cpu().numpy(), moment).astype(np.float32)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_sumsq(sizes, dt):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(n, generator=gen, device="cuda").to(tdt(dt)) for n in SIZES[sizes]]
    want = math.fsum(math.fsum(host(t) ** 2) for t in x)
    tl = zpq.TensorList(x)
    out = zpq.grad_sumsq(tl)
    # every addition rounds by 2^-53 at most; no element passes through more than
    # 2^16 of them here
    assert abs(out.item() - want) <= 2.0 ** -53 * 2 ** 16 * want
    again = zpq.grad_sumsq(tl)
    assert again.item() == out.item()
    zpq.grad_sumsq(tl, out=again, accumulate=True)
    assert again.item() == out.item() + out.item()


def test_sumsq_range():
    """Squares that binary32 cannot hold; infinities and NaN come through."""
    import torch
    x = torch.tensor([1e30, 2e30, 1e-30], device="cuda")
    want = sum(float(np.float32(v)) ** 2 for v in (1e30, 2e30, 1e-30))
    assert abs(zpq.grad_sumsq([x]).item() - want) <= 2.0 ** -51 * want
    assert zpq.grad_sumsq([torch.tensor([1.0, float("inf")], device="cuda")]).item() == math.inf
    assert math.isnan(zpq.grad_sumsq([torch.tensor([1.0, float("nan")], device="cuda")]).item())
    assert zpq.grad_sumsq([torch.empty(0, device="cuda")]).item() == 0.0


def test_new_gradients_and_other_stream():
    import torch
    d = make([5000, 77], bits=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    d0 = before(d)
    torch.cuda.synchronize()
    opt, total = run(d, 8, stream=side)
    side.synchronize()
    check(d0, d, 8, "f32", "bf16", total)
    d["g"] = [(g * 2).to(torch.float16) for g in d["g"]]
    opt.set_grads(d["g"])
    d0 = before(d)
    total = opt.grad_sumsq()
    opt.step(4, sumsq=total, max_norm=0.5)
    check(d0, d, 8, "f32", "bf16", total, step=4, max_norm=0.5)


def test_more_than_2_to_32_elements():
    """Offsets and random-number counters past 32 bits, in the last elements."""
    import torch
    n, tail = (1 << 32) + 300, 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    p[-tail:] = torch.randn(tail, generator=gen, device="cuda").bfloat16()
    g[-tail:] = torch.randn(tail, generator=gen, device="cuda").bfloat16()
    opt = zpq.AdamW([p], [g], state_bits=8, seed=7, weight_decay=0.1, **HYPER)
    total = opt.grad_sumsq()
    p0, g0 = host(p[-tail:]), host(g[-tail:])
    assert abs(total.item() - float((g0 ** 2).sum())) <= 2.0 ** -40 * total.item()
    opt.step(3, sumsq=total, max_norm=2.0)
    c = ref.clip_factor(total.item(), 1.0, 2.0)
    p1, _, _, tp, _, _ = ref.adamw64(p0, g0, np.zeros(tail), np.zeros(tail), c, HYPER["lr"], HYPER["betas"], HYPER["eps"], 0.1, 3)
    assert np.all(np.abs(host(p[-tail:]) - p1) <= tp + ref.HALF["bf16"] * (np.abs(p1) + tp) + ref.TINY["bf16"])
    first = (n - tail + 255) // 256 * 256                   # whole blocks from here on
    lead = first - (n - tail)
    ms, vs = ref.adamw32_moments(g0[lead:], np.zeros(tail - lead), np.zeros(tail - lead), c, HYPER["betas"])
    r = ref.random32(first, n - first, 7, 3)
    for x, moment, rnd, (codes, exps) in ((ms, 1, r & 0xFFFF, opt.exp_avg[0]), (vs, 2, r >> 16, opt.exp_avg_sq[0])):
        want_c, want_e = ref.encode8(x, moment, rnd)
        assert np.array_equal(exps[first // 256:].cpu().numpy(), want_e)
        assert np.array_equal(codes[first:].cpu().numpy(), want_c)
    assert not bool(p[: 1 << 20].any()) and not bool(opt.exp_avg_sq[0][0][: 1 << 20].any())


def test_random_numbers_cross_2_to_32_between_waves():
    """A tensor whose counters pass 2^32 in its third block, inside a part."""
    import torch
    big, n = (1 << 32) - 512, 2000
    gen = torch.Generator(device="cuda").manual_seed(3)
    p = [torch.zeros(big, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
    g = [torch.zeros(big, dtype=torch.bfloat16, device="cuda"),
         torch.randn(n, generator=gen, device="cuda").bfloat16()]
    opt = zpq.AdamW(p, g, state_bits=8, seed=11, **HYPER)
    opt.step(2)
    ms, vs = ref.adamw32_moments(host(g[1]), np.zeros(n), np.zeros(n), 1.0, HYPER["betas"])
    r = ref.random32(big, n, 11, 2)
    for x, moment, rnd, (codes, exps) in ((ms, 1, r & 0xFFFF, opt.exp_avg[1]), (vs, 2, r >> 16, opt.exp_avg_sq[1])):
        want_c, want_e = ref.encode8(x, moment, rnd)
        assert np.array_equal(exps.cpu().numpy(), want_e) and np.array_equal(codes.cpu().numpy(), want_c)


def test_captured_step_replays_equal_eager():
    import torch
    d, e = make([70000, 33], bits=8, seed=4), make([70000, 33], bits=8, seed=4)
    make_opt = lambda x: zpq.AdamW(x["p"], x["g"], copies=x["copy"], state_bits=8, exp_avg=x["m"],  # noqa: E731
                                   exp_avg_sq=x["v"], seed=3, **HYPER)
    od, oe = make_opt(d), make_opt(e)
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                      # warm-up, outside the capture
        od.grad_sumsq(out=total)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        od.grad_sumsq(out=total)
        od.step(5, sumsq=total, max_norm=1.0)
    gen = torch.Generator(device="cuda").manual_seed(8)
    for rep in range(4):
        print(f"graph replay {rep}", flush=True)
        for a, b in zip(d["g"], e["g"]):
            x = torch.randn(a.numel(), generator=gen, device="cuda").to(a.dtype)
            a.copy_(x)
            b.copy_(x)
        oe.step(5, sumsq=oe.grad_sumsq(), max_norm=1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in ("p", "copy"):
            assert all(torch.equal(a, b) for a, b in zip(d[k], e[k])), (rep, k)
        for k in ("m", "v"):
            assert all(torch.equal(a, b) for x, y in zip(d[k], e[k]) for a, b in zip(x, y)), (rep, k)


def test_refusals_on_the_gpu():
    import torch
    d = make([100, 20])
    ok = dict(copies=d["copy"], exp_avg=d["m"], exp_avg_sq=d["v"])
    with pytest.raises(ValueError):
        zpq.AdamW(d["p"], d["g"][:1], **ok)
    with pytest.raises(ValueError):
        zpq.AdamW(d["p"], [d["g"][0], d["g"][1][:-1]], **ok)
    with pytest.raises(ValueError):
        zpq.AdamW(d["p"], [d["g"][0], d["g"][1].float()], **ok)            # two types
    with pytest.raises(ValueError):
        zpq.AdamW(d["p"], d["g"], copies=[c.float() for c in d["copy"]])
    with pytest.raises(ValueError):
        zpq.AdamW(d["p"], d["g"], weight_decay=[0.1])
    with pytest.raises(ValueError):
        zpq.AdamW(d["p"], d["g"], state_bits=8, exp_avg=d["m"])
    with pytest.raises(ValueError):
        zpq.AdamW([d["p"][0].view(10, 10).t()], [d["g"][0]])               # not contiguous
    with pytest.raises(ValueError):
        zpq.AdamW(d["p"], d["g"], exp_avg=d["m"], exp_avg_sq=d["m"])       # one buffer twice
    with pytest.raises(ValueError):
        zpq.AdamW([d["p"][0], d["p"][0]], [d["g"][0], d["g"][0]])          # tied weights twice
    zpq.AdamW(d["p"], [d["g"][0], d["g"][0][:20]])                         # gradients are only read
    buf = torch.zeros(240, device="cuda")
    for at in (81, 99, 119):                                               # in the weights: both ends
        with pytest.raises(ValueError):
            zpq.AdamW([buf[100:120]], [buf[at:at + 20]])
    for at in (80, 120):                                                   # beside them
        zpq.AdamW([buf[100:120]], [buf[at:at + 20]])
    opt = zpq.AdamW(d["p"], d["g"], **ok)
    with pytest.raises(ValueError):
        opt.step(1, max_norm=1.0)
    with pytest.raises(ValueError):
        opt.step(1, sumsq=torch.zeros(1, device="cuda"))
    with pytest.raises(zpq.ZpqError):
        opt.step(0)
    with pytest.raises(zpq.ZpqError):
        zpq.state8_unpack(torch.zeros(5, dtype=torch.uint8, device="cuda"),
                          torch.zeros(1, dtype=torch.uint8, device="cuda"), 3)
