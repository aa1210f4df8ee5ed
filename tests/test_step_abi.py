"""The step operators without a GPU: argument checks of the C ABI and of the
binding (none of these calls launches anything), the structures' layout, and
the random numbers and 8-bit format of the definition."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import block_quantized_communication_amd as zpq
import step_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SIZE, BLOCK, ALIGN, DTYPE, MODE, LAUNCH, ARG, ALIAS = range(10)
P = 1 << 24                       # fake device addresses, never dereferenced
NUL = ctypes.c_void_p(0)
vp = ctypes.c_void_p


def arr(kind, values):
    return (kind * len(values))(*values)


def make_list(ptrs=(P, P + 4096), sizes=(10, 20), dtype=2, table=P + (1 << 20), nbytes=None, out=True):
    n = len(sizes)
    c = zpq._List()
    return zpq.lib().zpq_list_make(arr(vp, ptrs), arr(ctypes.c_int64, sizes), n, dtype, vp(table),
                                   n * 32 + 20736 if nbytes is None else nbytes,
                                   ctypes.byref(c) if out else None, NUL)


def test_list_refusals():
    assert make_list(dtype=3) == DTYPE
    assert make_list(sizes=(-1, 2)) == SIZE
    assert make_list(sizes=((1 << 40) + 1, 2)) == SIZE
    assert make_list(sizes=(1 << 40, 1)) == SIZE           # together
    assert make_list(ptrs=(0, P)) == NULL
    assert make_list(table=0) == NULL
    assert make_list(out=False) == NULL
    assert make_list(ptrs=(P + 1, P + 4096)) == ALIGN
    assert make_list(table=P + (1 << 20) + 8) == ALIGN
    assert make_list(nbytes=2 * 32 + 20735) == SIZE
    assert make_list(ptrs=(P, P + (1 << 20) + 16)) == ALIAS   # a tensor inside the table
    assert make_list(ptrs=(), sizes=(), table=0) == OK
    assert zpq.lib().zpq_list_make(None, None, -1, 0, NUL, 0, ctypes.byref(zpq._List()), NUL) == ARG


def sumsq(table=P, elems=100, chunks=1, count=1, dtype=0, out=P + (1 << 16)):
    c = zpq._List(table, elems, chunks, count, dtype)
    return zpq.lib().zpq_grad_sumsq(ctypes.byref(c), vp(out), 0, NUL)


def test_sumsq_refusals():
    assert zpq.lib().zpq_grad_sumsq(None, vp(P), 0, NUL) == NULL
    assert sumsq(dtype=9) == ARG
    assert sumsq(count=-1) == ARG
    assert sumsq(chunks=1 << 31) == ARG
    assert sumsq(table=0) == ARG
    assert sumsq(out=0) == NULL
    assert sumsq(out=P + (1 << 16) + 4) == ALIGN
    assert sumsq(out=P + 8) == ALIAS                        # in the table
    assert sumsq(out=P + 20736 + 24) == ALIAS


FIELDS = dict(p=P, g=P + 0x10000, m=P + 0x20000, v=P + 0x30000, m_exp=0, v_exp=0, copy=0, n=1000,
              weight_decay=0.0)


def plan(rows=None, count=None, pt=0, gt=2, ct=-1, bits=32, table=P + 0x100000, nbytes=None, out=True, **one):
    rows = [dict(FIELDS, **one)] if rows is None else rows
    t = arr(zpq._AdamwTensor, [zpq._AdamwTensor(**r) for r in rows])
    n = len(rows) if count is None else count
    c = zpq._AdamwPlan()
    return zpq.lib().zpq_adamw_plan_make(t, n, pt, gt, ct, bits, vp(table), n * 128 + 64 if nbytes is None else nbytes,
                                         ctypes.byref(c) if out else None, NUL)


def test_plan_refusals():
    assert plan(pt=5) == DTYPE
    assert plan(gt=-1) == DTYPE
    assert plan(ct=0) == DTYPE                                       # a copy in fp32
    assert plan(ct=1, pt=1) == MODE                                  # beside 16-bit weights
    assert plan(ct=1) == MODE                                        # announced, not given
    assert plan(copy=P + 0x40000) == MODE                            # given, not announced
    assert plan(bits=16) == ARG
    assert plan(weight_decay=-0.1) == ARG
    assert plan(weight_decay=float("nan")) == ARG
    assert plan(weight_decay=float("inf")) == ARG
    assert plan(n=-1) == SIZE
    assert plan(n=(1 << 40) + 1) == SIZE
    assert plan(rows=[dict(FIELDS, n=1 << 40), FIELDS]) == SIZE      # together
    for f in ("p", "g", "m", "v"):
        assert plan(**{f: 0}) == NULL, f
    assert plan(bits=8) == NULL                                      # no exponents
    assert plan(p=P + 2) == ALIGN
    assert plan(m=P + 0x20002) == ALIGN
    assert plan(g=P + 0x10001) == ALIGN
    assert plan(ct=2, copy=P + 0x40001) == ALIGN
    assert plan(table=P + 0x100008) == ALIGN
    assert plan(nbytes=191) == SIZE
    assert plan(m=P + 3996) == ALIAS                                 # the last bytes of p
    assert plan(g=P + 0x100010) == ALIAS                             # in the table
    assert plan(bits=8, m_exp=P + 0x50000, v_exp=P + 0x50003) == ALIAS
    assert plan(out=False) == NULL
    assert plan(table=0) == NULL
    assert plan(rows=[], table=0) == OK
    assert plan(rows=[], count=-1) == ARG


def step(count=1, chunks=1, table=P, bits=32, sumsq=None, **h):
    q = zpq._AdamwPlan(table, 100, chunks, count, 0, 2, -1, bits)
    v = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=1.0, max_norm=float("inf"), step=1, seed=0)
    return zpq.lib().zpq_adamw_step(ctypes.byref(q), ctypes.byref(zpq._AdamwHyper(**dict(v, **h))),
                                    vp(sumsq), NUL)


def test_step_refusals():
    nan, inf = float("nan"), float("inf")
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan),
                dict(beta2=1.0), dict(eps=0.0), dict(eps=nan), dict(eps=inf), dict(grad_scale=0.0),
                dict(grad_scale=nan), dict(grad_scale=inf), dict(max_norm=0.0), dict(max_norm=nan),
                dict(max_norm=1.0), dict(step=0), dict(bits=4), dict(table=0),
                dict(chunks=1 << 31), dict(count=-1)):
        assert step(**bad) == ARG, bad
    assert step(sumsq=P + 4) == ALIGN
    assert step(chunks=0) == OK
    assert zpq.lib().zpq_adamw_step(None, None, NUL, NUL) == NULL


def unpack(codes=P, exps=P + 0x10000, n=1000, moment=1, y=P + 0x20000, dt=0):
    return zpq.lib().zpq_state8_unpack(vp(codes), vp(exps), n, moment, vp(y), dt, NUL)


def pack(x=P + 0x20000, dt=0, n=1000, moment=2, codes=P, exps=P + 0x10000):
    return zpq.lib().zpq_state8_pack(vp(x), dt, n, moment, vp(codes), vp(exps), NUL)


@pytest.mark.parametrize("f,y", [(unpack, "y"), (pack, "x")])
def test_state8_refusals(f, y):
    assert f(moment=0) == ARG and f(moment=3) == ARG
    assert f(n=-1) == SIZE and f(n=(1 << 40) + 1) == SIZE
    assert f(dt=3) == DTYPE
    assert f(codes=0) == NULL and f(exps=0) == NULL and f(**{y: 0}) == NULL
    assert f(**{y: P + 0x20002}) == ALIGN
    assert f(**{y: P + 512}) == ALIAS
    assert f(exps=P + 999) == ALIAS
    assert f(n=0, codes=0, exps=0, **{y: 0}) == OK


def look(table=P, dt=1, rows=100, dim=16, ld=16, ids=P + 0x10000, ib=8, tokens=10, first=0, out=P + 0x20000, odt=1,
         lo=16):
    return zpq.lib().zpq_embedding(vp(table), dt, rows, dim, ld, vp(ids), ib, tokens, first, ctypes.c_float(1),
                                   vp(out), odt, lo, NUL)


def look8(codes=P, scales=P + 0x8000, rows=100, dim=16, block=32, ids=P + 0x10000, ib=4, tokens=10, out=P + 0x20000,
          odt=1, lo=16):
    return zpq.lib().zpq_embedding_i8(vp(codes), vp(scales), rows, dim, block, vp(ids), ib, tokens, 0,
                                      ctypes.c_float(1), vp(out), odt, lo, NUL)


@pytest.mark.parametrize("f", [look, look8])
def test_lookup_refusals(f):
    assert f(dim=0) == SIZE and f(rows=-1) == SIZE and f(tokens=-1) == SIZE
    assert f(rows=1 << 31) == SIZE and f(tokens=1 << 31) == SIZE
    assert f(lo=15) == SIZE and f(lo=1 << 41) == SIZE
    assert f(odt=3) == DTYPE
    assert f(ib=2) == ARG
    assert f(ids=0) == NULL and f(out=0) == NULL
    assert f(ids=P + 0x10002) == ALIGN and f(out=P + 0x20001) == ALIGN
    assert f(out=P + 64) == ALIAS and f(out=P + 0x10000 - 4) == ALIAS
    assert f(tokens=0, ids=0, out=0) == OK


def test_lookup_refusals_of_one_kind():
    assert look(dt=3) == DTYPE and look(ld=15) == SIZE and look(table=0) == NULL and look(table=P + 1) == ALIGN
    assert look8(block=48) == BLOCK and look8(block=0) == BLOCK and look8(block=1024) == BLOCK
    assert look8(codes=0) == NULL and look8(scales=0) == NULL and look8(scales=P + 0x8002) == ALIGN
    assert look8(out=P + 0x8000) == ALIAS


def grad(dy=P, dt=1, ldy=16, ids=P + 0x10000, ib=8, tokens=10, first=0, padding=-1, rows=100, dim=16,
         out=P + 0x20000, odt=0, lo=16, acc=0, ws=P + 0x40000, nbytes=1 << 20):
    return zpq.lib().zpq_embedding_grad(vp(dy), dt, ldy, vp(ids), ib, tokens, first, padding, rows, dim,
                                        ctypes.c_float(1), vp(out), odt, lo, acc, vp(ws), nbytes, NUL)


def test_grad_refusals():
    assert grad(dim=0) == SIZE and grad(rows=-1) == SIZE and grad(tokens=-1) == SIZE
    assert grad(rows=(1 << 27) + 1) == SIZE and grad(tokens=(1 << 28) + 1) == SIZE and grad(dim=(1 << 28) + 1) == SIZE
    assert grad(ldy=15) == SIZE and grad(lo=15) == SIZE
    assert grad(dt=3) == DTYPE and grad(odt=3) == DTYPE
    assert grad(ib=1) == ARG
    assert grad(out=0) == NULL and grad(dy=0) == NULL and grad(ids=0) == NULL and grad(ws=0) == NULL
    assert grad(nbytes=100) == SIZE
    assert grad(out=P + 0x20002) == ALIGN and grad(dy=P + 1) == ALIGN and grad(ids=P + 0x10004) == ALIGN
    assert grad(ws=P + 0x40008) == ALIGN
    assert grad(out=P + 64) == ALIAS and grad(ws=P + 0x20010) == ALIAS and grad(ws=P + 0x10010) == ALIAS
    assert grad(rows=0, out=0) == OK
    assert grad(tokens=0, acc=1) == OK
    n = ctypes.c_int64()
    assert zpq.lib().zpq_embedding_grad_bytes(10, 5, 16, None) == NULL
    assert zpq.lib().zpq_embedding_grad_bytes(-1, 5, 16, ctypes.byref(n)) == SIZE
    assert zpq.lib().zpq_embedding_grad_bytes(1, -1, 16, ctypes.byref(n)) == SIZE
    assert zpq.lib().zpq_embedding_grad_bytes(0, 5, 16, ctypes.byref(n)) == OK and 24 <= n.value <= 4096
    assert zpq.lib().zpq_embedding_grad_bytes(1 << 28, 5, 64, ctypes.byref(n)) == OK and n.value >= 2 << 31


def test_structures_match_the_header():
    """ctypes layouts against the C compiler's."""
    names = {"zpq_list": zpq._List, "zpq_adamw_tensor": zpq._AdamwTensor, "zpq_adamw_plan": zpq._AdamwPlan,
             "zpq_adamw_hyper": zpq._AdamwHyper}
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"zpq.h\"\nint main(void){\n"
    for n, s in names.items():
        src += f'printf("%zu", sizeof({n}));\n'
        for f, _ in s._fields_:
            src += f'printf(" %zu", offsetof({n}, {f}));\n'
        src += 'printf("\\n");\n'
    src += 'printf("%d %d\\n", (int)ZPQ_LIST_BYTES(3), (int)ZPQ_PLAN_BYTES(3)); return 0;}\n'
    exe = os.path.join(ROOT, "tests", "native", "step_layout.tmp")
    subprocess.run(["gcc", "-x", "c", "-", "-I", os.path.join(ROOT, "include"), "-o", exe], input=src, text=True, check=True)
    try:
        lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    finally:
        os.remove(exe)
    for line, s in zip(lines, names.values()):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert lines[-1] == f"{3 * 32 + zpq.LIST_FIXED_BYTES} {3 * 128 + 64}"


def test_binding_refuses_host_tensors():
    import torch
    x, i = torch.zeros(64), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: zpq.TensorList([x]), lambda: zpq.TensorList([]), lambda: zpq.grad_sumsq([x]),
                 lambda: zpq.AdamW([x], [x]), lambda: zpq.AdamW([], []), lambda: zpq.AdamW([x], [x], state_bits=16),
                 lambda: zpq.state8_unpack(x.byte(), x.byte(), 1), lambda: zpq.state8_pack(x, 1),
                 lambda: zpq.embedding(i, x.view(8, 8)), lambda: zpq.embedding_i8(i, x.char(), x, 8, 8),
                 lambda: zpq.embedding_grad(i, x.view(4, 16), 8)):
        with pytest.raises(ValueError):
            call()


def test_random_numbers_are_uniform_and_uncorrelated():
    """Halves of the hash over a million consecutive elements: 65536 cells of
    expectation 16 each; chi-squared / 65535 has deviation sqrt(2/65535) = 0.0055,
    and a correlation 0.001, so 6 deviations are 0.033 and 0.006."""
    for seed, step in ((0, 1), (1, 1), (12345, 999)):
        r = ref.random32(0, 1 << 20, seed, step)
        lo, hi = (r & 0xFFFF).astype(np.float64), (r >> 16).astype(np.float64)
        for a in (lo, hi):
            n = np.bincount(a.astype(np.int64), minlength=65536)
            assert abs(((n - 16.0) ** 2 / 16.0).sum() / 65535 - 1) < 0.033
            for gap in (1, 8, 64, 256, 2048):
                assert abs(np.corrcoef(a[:-gap], a[gap:])[0, 1]) < 0.006
        assert abs(np.corrcoef(lo, hi)[0, 1]) < 0.006
    across = ref.random32((1 << 32) - 4, 8, 3, 5)
    assert len(set(across.tolist())) == 8


@pytest.mark.parametrize("moment", [1, 2])
def test_eight_bit_format(moment):
    """Every code of the definition survives a round trip to nearest, and random
    rounding is unbiased and moves by one step at most."""
    n = 128 if moment == 1 else 256
    codes = np.zeros(256, np.uint8)
    codes[:n] = np.arange(n)
    if moment == 1:
        codes[128:] = np.arange(128) | 128
    exps = np.full(1, 130, np.uint8)
    x = ref.decode8(codes, exps, moment)
    assert x.astype(np.float32).astype(np.float64).tolist() == x.tolist()
    back, e = ref.encode8(x.astype(np.float32), moment)
    assert e[0] == 130 and np.array_equal(ref.decode8(back, e, moment), x)
    rng = np.random.default_rng(5)
    y = (rng.standard_normal(256) * 0.3).astype(np.float32)
    if moment == 2:
        y = np.abs(y)
    mean = np.zeros(256)
    trials = 400
    for t in range(trials):
        c, e = ref.encode8(y, moment, ref.random32(0, 256, t, 1) >> 16)
        mean += ref.decode8(c, e, moment) / trials
    # a step is at most 1/8 of the value (or of the smallest normal); the mean of
    # 400 draws deviates by at most step / 2 / 20, and 6 deviations of that are 0.15 steps
    step = np.maximum(np.abs(y), 2.0 ** -20) / 8
    assert np.all(np.abs(mean - y) < 0.15 * step + 1e-9)
