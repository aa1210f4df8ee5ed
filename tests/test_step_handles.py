"""The memory that the optimizer's and the norm's handles own: where new gradients
are written, on the CPU with a library that only takes note of the calls, and what
graphs and streams see of it on the GPU."""
import contextlib

import pytest

import block_quantized_communication_amd as zpq
from test_adamw import HYPER, make


class Calls:
    """Stands in for libzpq: notes each call's name and arguments."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        if not name.startswith("zpq_"):
            raise AttributeError(name)
        return lambda *args: self.made.append((name, args)) or 0


@pytest.fixture
def calls(monkeypatch):
    fake = Calls()
    monkeypatch.setattr(zpq, "lib", lambda: fake)
    monkeypatch.setattr(zpq, "_gpu", lambda t, name, device=None: t.device)
    monkeypatch.setattr(zpq, "_on", lambda stream, device: (0, contextlib.nullcontext()))
    monkeypatch.setattr("torch.cuda.current_stream", lambda device=None: None)
    return fake


def test_new_gradients_are_written_into_the_same_tables(calls):
    """A captured norm and step read both tables: neither may move or go while the
    optimizer lives.  Gradients of another type, which a captured kernel would read
    past their end or in half, leave the tables of the first type alone."""
    import torch
    p = [torch.zeros(10), torch.zeros(300)]
    opt = zpq.AdamW(p, [torch.zeros(10), torch.zeros(300)])
    at = {}
    for dt in (torch.float32, torch.float32, torch.bfloat16, torch.float16, torch.float32, torch.bfloat16):
        new = [torch.zeros(10, dtype=dt), torch.zeros(300, dtype=dt)]
        calls.made.clear()
        opt.set_grads(new)
        made = dict(calls.made)
        assert len(made) == len(calls.made) == 2
        assert list(made["zpq_list_make"][0]) == [g.data_ptr() for g in new]
        assert made["zpq_list_make"][3] == made["zpq_adamw_plan_make"][3] == zpq.dtype_code(dt)
        tables = (made["zpq_adamw_plan_make"][6], made["zpq_list_make"][4])
        assert at.setdefault(dt, tables) == tables
        assert all(a is b for a, b in zip(opt._list.tensors, new)) and opt.grads == opt._list.tensors
    assert len({t for pair in at.values() for t in pair}) == 6


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_norm_and_step_take_new_gradients(bits):
    """set_grads between the replays: each equals the eager step on the gradients
    that hold by then, while memory of the tables' sizes is allocated and written."""
    import torch
    sizes = [70000, 33]
    d, e = make(sizes, bits=bits, seed=4), make(sizes, bits=bits, seed=4)
    make_opt = lambda x: zpq.AdamW(x["p"], x["g"], copies=x["copy"], state_bits=bits, exp_avg=x["m"],  # noqa: E731
                                   exp_avg_sq=x["v"], seed=3, **HYPER)
    od, oe = make_opt(d), make_opt(e)
    table = od._list._table.data_ptr()
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
    flat = lambda x: [t for k in ("p", "copy", "m", "v") for y in x[k]  # noqa: E731
                      for t in (y if isinstance(y, tuple) else (y,))]
    for rep in range(4):
        print(f"graph replay {rep}", flush=True)
        new = [torch.randn(n, generator=gen, device="cuda").bfloat16() for n in sizes]
        od.set_grads(new)
        oe.set_grads(new)
        assert od._list._table.data_ptr() == table
        other = [torch.full((zpq.LIST_FIXED_BYTES + 64,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        want = oe.grad_sumsq()
        oe.step(5, sumsq=want, max_norm=1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(total, want), rep
        assert all(bool((x == 255).all()) for x in other), rep
        assert all(torch.equal(a, b) for a, b in zip(flat(d), flat(e))), rep
    print("another type, and a last replay", flush=True)
    od.set_grads([torch.zeros(n, device="cuda") for n in sizes])
    assert od.grad_sumsq().item() == 0.0
    want = oe.grad_sumsq()
    oe.step(5, sumsq=want, max_norm=1.0)               # on the gradients of the last round
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(total, want)
    assert all(torch.equal(a, b) for a, b in zip(flat(d), flat(e)))


@pytest.mark.parametrize("short", [True, False])
def test_the_current_stream_without_torch_s_short_way(short, monkeypatch):
    import torch
    stream = type("Stream", (), {"cuda_stream": 1234})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    if short:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    zpq._raw_stream.cache_clear()
    try:
        assert zpq._on(None, torch.device("cuda", 3))[0] == (1003 if short else 1234)
    finally:
        zpq._raw_stream.cache_clear()


class Memory:
    """A tensor that takes note of the streams it is recorded on."""

    def __init__(self):
        self.on = []

    def record_stream(self, s):
        self.on.append(s)


def test_memory_is_recorded_once_on_each_other_stream():
    home, other, third = (type("Stream", (), {"cuda_stream": i})() for i in (10, 11, 12))
    a, b = Memory(), Memory()
    held = zpq._Held()
    held.add([a], home.cuda_stream)
    for s in (home, other, other, third, home, third):
        held.used(s.cuda_stream, s, None)
    held.add([b], third.cuda_stream)                   # may be used on any of them from now on
    held.used(other.cuda_stream, other, None)
    assert a.on == [other, third] and b.on == [home, other]


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["list", "optimizer", "hyper"])
def test_handles_may_go_while_another_stream_uses_their_memory(what):
    """Made on the current stream, used on another that is still busy, dropped: the
    current stream's next allocations must not get that memory.  Nothing is written
    there meanwhile."""
    import torch
    n = 1 << 20
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    handle = zpq.TensorList([g]) if what == "list" else zpq.AdamW([p], [g])
    hyper = handle.device_hyper() if what == "hyper" else None
    mine = [handle._table] if what == "list" else \
        [hyper.data] if what == "hyper" else [handle.exp_avg[0], handle.exp_avg_sq[0]] + \
        [t for table, made in handle._tables.values() for t in (table, made._table)]
    sizes = [t.numel() * t.element_size() for t in mine]
    at = {t.untyped_storage().data_ptr() for t in mine}
    del mine
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)                 # some tenths of a second
        if what == "hyper":
            handle.step(hyper)
        elif what == "optimizer":
            handle.step(1, sumsq=handle.grad_sumsq(out=total))
        else:
            zpq.grad_sumsq(handle, out=total)
    del hyper
    if what != "hyper":
        del handle
    new = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(4)]
    busy = not side.query()
    got = {t.untyped_storage().data_ptr() for t in new}
    torch.cuda.synchronize()
    assert busy, "the other stream had ended: nothing was tested"
    assert not at & got
