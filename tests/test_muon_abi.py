"""Orthogonalisation and the Muon step without a GPU: argument checks of the C ABI and of the binding
(none of these calls launches anything) and the structures' layout."""
import ctypes
import os
import subprocess

import pytest
import torch

import block_quantized_communication_amd as zpq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SIZE, BLOCK, ALIGN, DTYPE, MODE, LAUNCH, ARG, ALIAS = range(10)
P = 1 << 28                       # fake device addresses, never dereferenced
MB = 1 << 20
INF = float("inf")
C = (ctypes.c_double * 6)(3.4445, -4.775, 2.0315, 1.5, -0.5, 0.0)


def ortho(x=P, dt=0, count=3, rows=100, cols=200, ld=200, apart=20000, coeffs=C, steps=2, out=P + 8 * MB, ot=2, lo=200, ao=20000,
          ws=P + 16 * MB, nbytes=64 * MB):
    return zpq.lib().zpq_orthogonalize(x, dt, count, rows, cols, ld, apart, coeffs, steps, out, ot, lo, ao, ws, nbytes, None)


def test_orthogonalize_refusals():
    assert ortho(dt=3) == DTYPE and ortho(ot=0) == DTYPE and ortho(ot=5) == DTYPE
    assert ortho(coeffs=None) == NULL
    assert ortho(steps=0) == ARG and ortho(steps=33) == ARG
    for bad in (float("nan"), INF, 65.0):
        assert ortho(coeffs=(ctypes.c_double * 3)(1.0, bad, 1.0), steps=1) == ARG
    assert ortho(count=-1) == SIZE and ortho(count=(1 << 20) + 1) == SIZE
    assert ortho(rows=-1) == SIZE and ortho(cols=(1 << 22) + 1) == SIZE
    assert ortho(rows=1 << 20, cols=1 << 20) == SIZE
    assert ortho(ld=199) == SIZE and ortho(lo=100) == SIZE
    assert ortho(apart=19999) == SIZE and ortho(ao=0) == SIZE
    assert ortho(x=0) == NULL and ortho(out=0) == NULL and ortho(ws=0) == NULL
    need = ctypes.c_int64()
    assert zpq.lib().zpq_orthogonalize_bytes(3, 100, 200, ctypes.byref(need)) == OK
    assert zpq.lib().zpq_orthogonalize_bytes(3, 100, 200, None) == NULL
    assert zpq.lib().zpq_orthogonalize_bytes(3, -1, 200, ctypes.byref(ctypes.c_int64())) == SIZE
    assert ortho(nbytes=need.value - 1) == SIZE
    assert ortho(x=P + 2) == ALIGN and ortho(out=P + 8 * MB + 1) == ALIGN and ortho(ws=P + 16 * MB + 128) == ALIGN
    assert ortho(out=P + 239984) == ALIAS and ortho(ws=P) == ALIAS and ortho(ws=P + 8 * MB) == ALIAS
    assert ortho(count=0) == OK and ortho(rows=0) == OK and ortho(cols=0) == OK


def test_workspace_is_bounded():
    need = ctypes.c_int64()
    assert zpq.lib().zpq_orthogonalize_bytes(1000, 1024, 1024, ctypes.byref(need)) == OK
    assert need.value < 20 << 26                           # of 2^26 elements, not of all


FIELDS = dict(p=P, g=P + MB, m=P + 2 * MB, copy=0, rows=100, cols=200, weight_decay=0.0, scale=1.0)


def plan(pt=0, gt=2, ct=-1, memory=P + 8 * MB, nbytes=64 * MB, out=True, count=1, **one):
    rows = (zpq._MuonMatrix * 1)(zpq._MuonMatrix(**dict(FIELDS, **one)))
    c = zpq._MuonPlan()
    return zpq.lib().zpq_muon_plan_make(rows, count, pt, gt, ct, memory, nbytes, ctypes.byref(c) if out else None, None)


def test_plan_refusals():
    assert plan(pt=3) == DTYPE and plan(gt=-1) == DTYPE and plan(ct=0) == DTYPE
    assert plan(pt=1, ct=1) == MODE                                  # a copy beside 16-bit weights
    assert plan(ct=1) == MODE and plan(copy=P + 3 * MB) == MODE
    assert plan(out=False) == NULL and plan(memory=0) == NULL
    assert plan(p=0) == NULL and plan(g=0) == NULL and plan(m=0) == NULL
    assert plan(count=-1) == ARG
    for bad in (-1.0, float("nan"), INF):
        assert plan(weight_decay=bad) == ARG and plan(scale=bad) == ARG
    assert plan(rows=-1) == SIZE and plan(rows=1 << 18, cols=1 << 18) == SIZE and plan(nbytes=100) == SIZE
    assert plan(p=P + 2) == ALIGN and plan(g=P + MB + 1) == ALIGN and plan(m=P + 2 * MB + 2) == ALIGN
    assert plan(ct=2, copy=P + 3 * MB + 1) == ALIGN and plan(memory=P + 8 * MB + 16) == ALIGN
    assert plan(g=P + 79984) == ALIAS and plan(m=P + 16) == ALIAS and plan(ct=2, copy=P + 2 * MB) == ALIAS
    assert plan(memory=P) == ALIAS
    need = ctypes.c_int64()
    rows = (zpq._MuonMatrix * 1)(zpq._MuonMatrix(**FIELDS))
    assert zpq.lib().zpq_muon_plan_bytes(rows, 1, None) == NULL
    assert zpq.lib().zpq_muon_plan_bytes(None, 1, ctypes.byref(need)) == NULL
    assert zpq.lib().zpq_muon_plan_bytes(None, 0, ctypes.byref(need)) == OK
    assert zpq.lib().zpq_muon_plan_make(None, 0, 0, 0, -1, None, 64 + 192, ctypes.byref(zpq._MuonPlan()), None) == OK


def step(plan=None, sumsq=None, coeffs=C, hyper=True, **kw):
    h = dict(lr=0.1, momentum=0.9, grad_scale=1.0, max_norm=INF, steps=2, nesterov=1)
    h.update(kw)
    rows = (zpq._MuonMatrix * 1)(zpq._MuonMatrix(**FIELDS))
    p = zpq._MuonPlan(P, rows, 0, 0, 2, -1) if plan is None else plan
    x = zpq._MuonHyper(h["lr"], h["momentum"], h["grad_scale"], h["max_norm"], coeffs, h["steps"], h["nesterov"])
    return zpq.lib().zpq_muon_step(ctypes.byref(p), ctypes.byref(x) if hyper else None, sumsq, None)


def test_step_refusals():
    assert step() == OK                                    # a plan of no matrices
    assert zpq.lib().zpq_muon_step(None, None, None, None) == NULL
    assert step(hyper=False) == NULL and step(coeffs=None) == NULL
    for bad in (-0.1, float("nan"), INF):
        assert step(lr=bad) == ARG
        assert step(momentum=bad) == ARG
    assert step(momentum=1.0) == ARG
    for bad in (0.0, -1.0, INF, float("nan")):
        assert step(grad_scale=bad) == ARG
    assert step(max_norm=0.0) == ARG and step(max_norm=float("nan")) == ARG
    assert step(max_norm=1.0) == ARG                       # without a norm
    assert step(max_norm=1.0, sumsq=P + 4) == ALIGN
    assert step(steps=0) == ARG and step(steps=40) == ARG
    rows = (zpq._MuonMatrix * 1)(zpq._MuonMatrix(**FIELDS))
    assert step(plan=zpq._MuonPlan(P, rows, -1, 0, 2, -1)) == ARG
    assert step(plan=zpq._MuonPlan(None, rows, 1, 0, 2, -1)) == ARG
    assert step(plan=zpq._MuonPlan(P, rows, 1, 7, 2, -1)) == ARG


def test_binding_refusals():
    m = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="GPU"):
        zpq.orthogonalize(m)
    with pytest.raises(ValueError, match="GPU"):
        zpq.Muon([m], [m])
    with pytest.raises(ValueError, match="at least one"):
        zpq.Muon([], [])
    with pytest.raises(ValueError, match="coeffs"):
        zpq._coeffs_of((1.0, 2.0), 5)
    with pytest.raises(ValueError, match="coeffs"):
        zpq._coeffs_of(((1.0, 2.0, 3.0),) * 4, 5)
    assert list(zpq._coeffs_of((1, 2, 3), 2)[0]) == [1, 2, 3, 1, 2, 3]
    cpu = torch.device("cpu")
    assert zpq._stack(torch.zeros(3, 4, 6)[:, 1:3, 2:5], "x", cpu) == (3, 2, 3, 6, 24)
    assert zpq._stack(torch.zeros(1, 4, 6), "x", cpu) == (1, 4, 6, 6, 24)
    with pytest.raises(ValueError, match="overlap"):
        zpq._stack(torch.zeros(4, 6).expand(3, 4, 6), "x", cpu)
    with pytest.raises(ValueError, match="overlap"):
        zpq._stack(torch.zeros(3, 6, 4).transpose(1, 2), "x", cpu)
    with pytest.raises(ValueError, match="2-D or 3-D"):
        zpq._stack(torch.zeros(5), "x", cpu)


@pytest.mark.parametrize("name,cls", [("zpq_muon_matrix", "_MuonMatrix"), ("zpq_muon_plan", "_MuonPlan"), ("zpq_muon_hyper", "_MuonHyper")])
def test_struct_layout(name, cls, tmp_path):
    cls = getattr(zpq, cls)
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "zpq.h"\nint main(void) {\n' +
                   "".join(f'printf("%zu ", offsetof({name}, {f}));\n' for f in fields) + f'printf("%zu", sizeof({name})); return 0; }}\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls)]
