"""The 8-bit floating-point operators without a GPU: argument checks of the C ABI and of the binding
(none of these calls launches anything), the structure's layout, and the definition's own numbers."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import block_quantized_communication_amd as zpq
import float8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SIZE, BLOCK, ALIGN, DTYPE, MODE, LAUNCH, ARG, ALIAS = range(10)
P = 1 << 28                       # fake device addresses, never dereferenced
MB = 1 << 20


def quant(x=P, dt=2, rows=100, cols=300, ld=300, kind=0, tile=0, codes=P + MB, scales=P + 2 * MB, codes_t=P + 3 * MB,
          scales_t=P + 4 * MB):
    return zpq.lib().zpq_quant_f8(x, dt, rows, cols, ld, kind, tile, codes, scales, codes_t, scales_t, None)


def test_quant_refusals():
    assert quant(dt=3) == DTYPE
    assert quant(kind=2) == DTYPE
    assert quant(rows=-1) == SIZE
    assert quant(cols=-1) == SIZE
    assert quant(ld=299) == SIZE
    assert quant(rows=1 << 21, cols=1 << 20, ld=1 << 20) == SIZE
    assert quant(rows=2, cols=(1 << 23) + 1, ld=(1 << 23) + 1, codes_t=0, scales_t=0) == SIZE     # a row of codes over 2^23
    assert quant(rows=(1 << 23) + 1, cols=1, ld=1) == SIZE
    assert quant(rows=1 << 28, cols=1, ld=1, codes_t=0, scales_t=0) == SIZE                       # blocks
    assert quant(rows=1 << 20, cols=1 << 20, ld=1 << 20) == SIZE                                  # tiles
    assert quant(codes=0) == MODE
    assert quant(scales_t=0) == MODE
    assert quant(codes=0, scales=0, codes_t=0, scales_t=0) == MODE
    assert quant(x=0) == NULL
    assert quant(x=P + 1) == ALIGN
    for name in ("codes", "scales", "codes_t", "scales_t"):
        assert quant(**{name: P + 8 * MB + 8}) == ALIGN
    assert quant(codes=P + 59984) == ALIAS                 # 100 x 300 bf16: 60,000 bytes
    assert quant(scales=P + MB + 100 * 384 - 16) == ALIAS
    assert quant(scales_t=P + 3 * MB + 300 * 128 - 16) == ALIAS
    assert quant(rows=0) == OK and quant(cols=0, codes=0, scales=0, codes_t=0, scales_t=0) == OK


def dequant(codes=P, kind=0, scales=P + MB, rows=100, cols=300, tile=0, y=P + 2 * MB, dt=0, ld=300):
    return zpq.lib().zpq_dequant_f8(codes, kind, scales, rows, cols, tile, y, dt, ld, None)


def test_dequant_refusals():
    assert dequant(dt=7) == DTYPE
    assert dequant(kind=-1) == DTYPE
    assert dequant(rows=-1) == SIZE
    assert dequant(cols=(1 << 23) + 1) == SIZE
    assert dequant(ld=200) == SIZE
    assert dequant(rows=1 << 28, cols=1, ld=1) == SIZE
    assert dequant(codes=0) == NULL and dequant(scales=0) == NULL and dequant(y=0) == NULL
    assert dequant(codes=P + 8) == ALIGN and dequant(scales=P + MB + 4) == ALIGN and dequant(y=P + 2 * MB + 2) == ALIGN
    assert dequant(y=P + 100 * 384 - 16) == ALIAS and dequant(y=P + MB + 396) == ALIAS
    assert dequant(rows=0) == OK and dequant(cols=0) == OK


def transpose(codes=P, scales=P + MB, rows=100, cols=300, codes_t=P + 2 * MB, scales_t=P + 3 * MB):
    return zpq.lib().zpq_transpose_f8(codes, scales, rows, cols, codes_t, scales_t, None)


def test_transpose_refusals():
    assert transpose(rows=-1) == SIZE and transpose(cols=(1 << 23) + 1) == SIZE
    assert transpose(rows=1 << 20, cols=1 << 20) == SIZE
    for name in ("codes", "scales", "codes_t", "scales_t"):
        assert transpose(**{name: 0}) == NULL
        assert transpose(**{name: P + 8 * MB + 8}) == ALIGN
    assert transpose(codes_t=P + 100 * 384 - 16) == ALIAS
    assert transpose(scales_t=P + 2 * MB) == ALIAS
    assert transpose(rows=0) == OK


def matmul(m=100, n=200, k=1000, out=P + 8 * MB, dt=2, ld=200, accumulate=0, ws=P + 16 * MB, nbytes=None, a=None, b=None, **one):
    at = dict(a_codes=P, a_scales=P + MB, a_kind=0, a_tile=0, b_codes=P + 2 * MB, b_scales=P + 3 * MB, b_kind=1, b_tile=1)
    at.update(one)
    oa, ob = (zpq._F8(at[s + "codes"], at[s + "scales"], at[s + "kind"], at[s + "tile"]) for s in ("a_", "b_"))
    if nbytes is None:
        need = ctypes.c_int64()
        nbytes = need.value if zpq.lib().zpq_matmul_f8_bytes(m, n, k, ctypes.byref(need)) == 0 else 0
        nbytes = need.value
    return zpq.lib().zpq_matmul_f8(None if a == 0 else oa, None if b == 0 else ob, m, n, k, out, dt, ld, accumulate, ws, nbytes, None)


def test_matmul_refusals():
    assert matmul(a=0) == NULL and matmul(b=0) == NULL
    assert matmul(dt=4) == DTYPE and matmul(a_kind=2) == DTYPE and matmul(b_kind=-1) == DTYPE
    for name in ("m", "n", "k"):
        assert matmul(**{name: -1}) == SIZE
    assert matmul(k=(1 << 23) + 1) == SIZE
    assert matmul(m=1 << 31, n=1, ld=1) == SIZE and matmul(n=1 << 31, m=1) == SIZE
    assert matmul(m=1 << 20, n=1 << 20, ld=1 << 20) == SIZE
    assert matmul(ld=199) == SIZE
    assert matmul(out=0) == NULL
    for name in ("a_codes", "a_scales", "b_codes", "b_scales"):
        assert matmul(**{name: 0}) == NULL
        assert matmul(**{name: P + 32 * MB + 8}) == ALIGN
    assert matmul(out=P + 8 * MB + 1) == ALIGN
    assert matmul(out=P + 100 * 1024 - 16) == ALIAS        # in a's codes
    assert matmul(out=P + 3 * MB + 8) == ALIAS             # in b's scales
    assert matmul(m=0) == OK and matmul(n=0, ld=0) == OK
    assert matmul(m=0, out=0, a_codes=0, b_scales=0) == OK
    assert matmul(k=0, accumulate=1, a_codes=0, b_scales=0, a_scales=0, b_codes=0) == OK
    need = ctypes.c_int64()
    assert zpq.lib().zpq_matmul_f8_bytes(1, 2, 3, None) == NULL
    assert zpq.lib().zpq_matmul_f8_bytes(-1, 2, 3, ctypes.byref(need)) == SIZE
    assert zpq.lib().zpq_matmul_f8_bytes(64, 64, 1 << 20, ctypes.byref(need)) == OK and need.value > 0
    big = dict(m=64, n=64, ld=64, k=1 << 20, a_codes=P, b_codes=P + 128 * MB, a_scales=P + 256 * MB, b_scales=P + 272 * MB,
               out=P + 288 * MB, ws=P + 300 * MB)
    assert matmul(**{**big, "ws": 0}) == NULL
    assert matmul(**big, nbytes=need.value - 1) == SIZE
    assert matmul(**{**big, "ws": P + 300 * MB + 8}) == ALIGN
    assert matmul(**{**big, "ws": P + 64}) == ALIAS
    assert matmul(**{**big, "ws": P + 288 * MB}) == ALIAS


def test_binding_refusals():
    """Everything that can be refused without a GPU is."""
    x = torch.zeros(4, 256)
    codes, scales = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(4, 4, dtype=torch.uint8)
    for call in (lambda: zpq.quant_f8(x), lambda: zpq.quant_f8(x, along="both"), lambda: zpq.dequant_f8(codes, scales),
                 lambda: zpq.transpose_f8(codes, scales), lambda: zpq.matmul_f8((codes, scales), (codes, scales))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="along"):
        zpq.quant_f8(x, along="tile")
    with pytest.raises(ValueError, match="3 blocks"):
        zpq._f8_cols(256, 3, "cols")
    assert zpq._f8_cols(257, 3, "cols") == 257 and zpq._f8_cols(None, 3, "cols") == 384
    with pytest.raises(ValueError, match="float8"):
        zpq._kind(torch.int8, "codes")


def test_struct_layout(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "zpq.h"\n#define P(f) printf("%zu ", offsetof(zpq_f8_operand, f))\n'
                   'int main(void) { P(codes); P(scales); P(kind); P(tile); printf("%zu", sizeof(zpq_f8_operand)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    f = zpq._F8
    assert got == [f.codes.offset, f.scales.offset, f.kind.offset, f.tile.offset, ctypes.sizeof(f)]


@pytest.mark.parametrize("kind,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_reference_codes(kind, dtype):
    """The tests' own tables against torch's conversions, which are another implementation."""
    every = torch.arange(256, dtype=torch.uint8)
    want = every.view(dtype).double().numpy()
    got = ref.decode(every.numpy(), kind)
    fine = np.isfinite(want)
    assert np.array_equal(got[fine], want[fine]) and not np.isfinite(got[~fine]).any()
    rng = np.random.default_rng(0)
    top = 1.75 * 2.0 ** ref.TOP[kind]
    x = np.concatenate([rng.uniform(-top, top, 20000), rng.standard_normal(20000) * 2.0 ** rng.integers(-20, 5, 20000)])
    x = x.astype(np.float32).astype(np.float64)
    mid = ref.table(kind)
    mid = mid[np.isfinite(mid)]
    x = np.concatenate([x, (mid[1:] + mid[:-1]) / 2, -(mid[1:] + mid[:-1]) / 2])
    assert np.array_equal(ref.encode(x, kind), torch.from_numpy(x).float().to(dtype).view(torch.uint8).numpy())
