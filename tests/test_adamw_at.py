"""The optimizer step with its hyperparameters in device memory: the same bits as
with host ones, for every number of steps, and in a replayed graph that counts
its own steps."""
import ctypes

import pytest

import block_quantized_communication_amd as zpq
from test_adamw import HYPER, make

NULL, ALIGN, ARG, ALIAS, OK = 1, 4, 8, 9, 0
P = 0x7F0000000000                                     # addresses that no test reads
vp = ctypes.c_void_p


def at(h=P, sumsq=None, count=1, chunks=1, table=P + 0x100000, bits=32, plan=True):
    q = zpq._AdamwPlan(table, 100, chunks, count, 0, 2, -1, bits)
    return zpq.lib().zpq_adamw_step_at(ctypes.byref(q) if plan else None, vp(h), vp(sumsq), vp(None))


def test_refusals_without_a_gpu():
    assert at(plan=False) == NULL
    assert at(h=None) == NULL
    assert at(h=P + 4) == ALIGN
    assert at(sumsq=P + 4) == ALIGN
    assert at(h=P + 0x100000 + 184) == ALIAS           # the last 8 bytes of the plan's table
    assert at(h=P + 0x100000 - 56) == ALIAS
    for bad in (dict(bits=4), dict(table=0), dict(count=-1), dict(count=0), dict(chunks=-1), dict(chunks=1 << 31)):
        assert at(**bad) == ARG, bad
    assert at(chunks=0) == OK


def pair(sizes, bits, **kw):
    d, e = make(sizes, bits=bits, **kw), make(sizes, bits=bits, **kw)
    opt = lambda x: zpq.AdamW(x["p"], x["g"], copies=x["copy"], state_bits=bits, exp_avg=x["m"],  # noqa: E731
                              exp_avg_sq=x["v"], seed=3, weight_decay=0.1, **HYPER)
    return d, e, opt(d), opt(e)


def all_equal(d, e, what):
    import torch
    flat = lambda x: [t for k in ("p", "copy", "m", "v") for y in x[k] or ()  # noqa: E731
                      for t in (y if isinstance(y, tuple) else (y,))]
    assert all(torch.equal(a, b) for a, b in zip(flat(d), flat(e))), what


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[1], [700, 0, 33], [1 + i * 37 % 300 for i in range(70)]], ids=["one", "three", "many"])
def test_same_bits_as_host_hyperparameters(sizes, bits):
    d, e, od, oe = pair(sizes, bits)
    h = od.device_hyper(max_norm=0.5)
    for step, lr, scale in ((1, 3e-3, 1.0), (2, 1e-3, 0.125), (3, 0.0, 1.0), (1000, 2e-3, 4.0), (1 << 40, 1e-3, 1.0)):
        h.step.fill_(step)
        h.lr.fill_(lr)
        h.grad_scale.fill_(scale)
        od.step(h, sumsq=od.grad_sumsq())
        oe.step(step, lr=lr, grad_scale=scale, sumsq=oe.grad_sumsq(), max_norm=0.5)
        all_equal(d, e, step)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_out_of_range_changes_nothing(bits):
    d, e, od, _ = pair([300, 5], bits)
    nan, inf = float("nan"), float("inf")
    for field, bad in (("step", 0), ("step", -3), ("lr", -1.0), ("lr", nan), ("lr", inf), ("grad_scale", 0.0),
                       ("grad_scale", nan), ("max_norm", 0.0), ("max_norm", nan)):
        h = od.device_hyper(max_norm=1.0)
        getattr(h, field).fill_(bad)
        od.step(h, sumsq=od.grad_sumsq())
        all_equal(d, e, (field, bad))


@pytest.mark.gpu
def test_without_a_norm_and_refusals():
    d, e, od, oe = pair([4097, 12], 32)
    od.step(od.device_hyper(step=4, grad_scale=0.5))
    oe.step(4, grad_scale=0.5)
    all_equal(d, e, "no norm")
    h = od.device_hyper(max_norm=1.0)
    with pytest.raises(ValueError):
        od.step(h)
    for kw in (dict(lr=1e-3), dict(grad_scale=2.0), dict(max_norm=1.0)):
        with pytest.raises(ValueError):
            od.step(h, sumsq=od.grad_sumsq(), **kw)
    all_equal(d, e, "refusals")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_captured_graph_counts_its_steps(bits):
    import torch
    d, e, od, oe = pair([70000, 33], bits, seed=4)
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    h = od.device_hyper(step=4, max_norm=1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                      # warm-up, outside the capture
        od.grad_sumsq(out=total)
        h.step.add_(0)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.step.add_(1)
        od.grad_sumsq(out=total)
        od.step(h, sumsq=total)
    gen = torch.Generator(device="cuda").manual_seed(8)
    for rep in range(5):
        print(f"graph replay {rep}", flush=True)
        for a, b in zip(d["g"], e["g"]):
            x = torch.randn(a.numel(), generator=gen, device="cuda").to(a.dtype)
            a.copy_(x)
            b.copy_(x)
        h.lr.fill_(1e-3 / (1 + rep))
        oe.step(5 + rep, lr=1e-3 / (1 + rep), sumsq=oe.grad_sumsq(), max_norm=1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert h.step.item() == 5 + rep
        all_equal(d, e, rep)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_without_a_norm_max_norm_is_not_looked_at(bits):
    """And it is, whenever it is written, where the step gets a norm."""
    d, e, od, oe = pair([4097, 12], bits)
    h = od.device_hyper(step=4)
    for i, x in enumerate((0.0, -1.0, float("nan"), 1e-3)):
        h.max_norm.fill_(x)
        h.step.fill_(4 + i)
        od.step(h)
        oe.step(4 + i)
        all_equal(d, e, x)
    od.step(h, sumsq=od.grad_sumsq())
    oe.step(7, sumsq=oe.grad_sumsq(), max_norm=1e-3)
    all_equal(d, e, "clipped")
