"""CPU tests of libue5m3fp4_layer's refusals: the C ABI rejects bad arguments
on the host before any HIP call (the pointers are never dereferenced), and the
Python binding rejects malformed operands before it takes a pointer (the
stand-ins of test_binding_checks fail if their address is requested)."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import fp4_block_scaled_amax_amd as lib
from test_binding_checks import Dev, raises

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ue5m3fp4_layer.h")
OK, EINVAL, ESHAPE, EALIGN, ERANGE = 0, -1, -2, -3, -5
P = 0x10000


@pytest.fixture(scope="module")
def L():
    return lib.load_layer_library()


def test_exports_and_c99_header(L, tmp_path):
    names = sorted(re.findall(r"UE5M3FP4_API\s+int\s+(ue5m3fp4_\w+)\(", open(HEADER).read()))
    out = subprocess.run(["nm", "-D", "--defined-only", lib.LAYER_LIB_PATH], capture_output=True, text=True).stdout
    assert sorted(re.findall(r" T (\S+)", out)) == names
    gcc = shutil.which("gcc")
    if gcc:
        src = tmp_path / "a.c"
        src.write_text('#include "ue5m3fp4_layer.h"\nint main(void) { return UE5M3FP4_E5M2 + UE5M3FP4_F32 - 2; }\n')
        subprocess.run([gcc, "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-c", str(src), "-o", str(tmp_path / "a.o")], check=True)


def qz(L, x=P, rows=32, cols=32, ld=32, fmt=0, st=0, tile=0, rc=P, rs=P, cc=2 * P, cs=2 * P):
    return L.ue5m3fp4_quantize_fp8(x, rows, cols, ld, fmt, st, tile, rc, rs, cc, cs, None)


def test_quantize_argument_checks(L):
    assert qz(L, rows=-1) == EINVAL
    assert qz(L, fmt=2) == EINVAL and qz(L, st=2) == EINVAL and qz(L, tile=2) == EINVAL
    assert qz(L, x=None) == EINVAL
    assert qz(L, rc=None) == EINVAL and qz(L, cs=None) == EINVAL
    assert qz(L, rc=None, rs=None, cc=None, cs=None) == EINVAL
    assert qz(L, cc=P) == EINVAL and qz(L, cs=P) == EINVAL  # one buffer for both outputs
    assert qz(L, ld=31) == ESHAPE
    assert qz(L, x=P + 8) == EALIGN and qz(L, rc=P + 8) == EALIGN and qz(L, rs=P + 4) == EALIGN
    assert qz(L, rows=1 << 31) == ERANGE and qz(L, cols=1 << 31, ld=1 << 31) == ERANGE
    assert qz(L, rows=(1 << 31) - 1, ld=1 << 39) == ERANGE
    assert qz(L, rows=0, x=None) == OK and qz(L, cols=0, ld=0, x=None) == OK


def gm(L, ac=P, as_=P, af=0, at=0, bc=P, bs=P, bf=0, bt=0, st=0, M=32, N=32, K=32, c=P, ct=0):
    return L.ue5m3fp4_gemm_fp8_nt(ac, as_, af, at, bc, bs, bf, bt, st, M, N, K, c, ct, None)


def test_gemm_argument_checks(L):
    assert gm(L, M=-1) == EINVAL and gm(L, K=-1) == EINVAL
    for k in ("af", "at", "bf", "bt", "st", "ct"):
        assert gm(L, **{k: 2}) == EINVAL and gm(L, **{k: -1}) == EINVAL
    for k in ("ac", "as_", "bc", "bs", "c"):
        assert gm(L, **{k: None}) == EINVAL
        assert gm(L, **{k: P + 8}) == EALIGN
    assert gm(L, K=1 << 24) == ERANGE
    assert gm(L, M=1 << 31) == ERANGE and gm(L, M=1 << 20, N=1 << 20) == ERANGE
    assert gm(L, M=(1 << 31) - 1, N=1, K=1 << 10) == ERANGE
    assert gm(L, M=0, c=None) == OK and gm(L, N=0, c=None) == OK


def dr(L, x=P, xt=0, ldx=32, r=None, ldr=0, o=P, ot=0, ldo=32, rows=8, cols=32, p=0.5, amax=None):
    return L.ue5m3fp4_dropout(x, xt, ldx, r, ldr, o, ot, ldo, rows, cols, p, 0, 0, amax, None)


def test_dropout_argument_checks(L):
    assert dr(L, rows=-1) == EINVAL and dr(L, xt=2) == EINVAL and dr(L, ot=-1) == EINVAL
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert dr(L, p=p) == EINVAL
    assert dr(L, x=None) == EINVAL and dr(L, o=None) == EINVAL
    assert dr(L, ldx=31) == ESHAPE and dr(L, ldo=31) == ESHAPE and dr(L, r=P, ldr=31) == ESHAPE
    assert dr(L, r=P, ldr=-1) == EINVAL
    assert dr(L, x=P + 8) == EALIGN and dr(L, o=P + 2) == EALIGN and dr(L, r=P + 4, ldr=32) == EALIGN
    assert dr(L, amax=P + 2) == EALIGN
    assert dr(L, rows=1 << 31) == ERANGE and dr(L, rows=1 << 20, ldx=1 << 20) == ERANGE
    assert dr(L, rows=0, x=None) == OK and dr(L, cols=0, x=None) == OK
    f = L.ue5m3fp4_dropout_backward
    assert f(P, 0, 32, P, 0, 32, 8, 32, 2.0, 0, 0, None, None) == EINVAL
    assert f(None, 0, 32, P, 0, 32, 8, 32, 0.5, 0, 0, None, None) == EINVAL


def t(*shape, dtype=torch.float32):
    return Dev(torch.zeros(shape, dtype=dtype))


def operand(rows, cols, fmt=lib.E4M3, e8m0=False, tile=False):
    q = lib.empty_quantized_fp8(rows, cols, fmt, e8m0, tile, device="cpu")
    return lib.Fp8Quantized(Dev(q.codes), Dev(q.scales), cols, fmt, tile)


def test_operand_shapes():
    q = lib.empty_quantized_fp8(300, 130, lib.E5M2, True, True, device="cpu")
    assert q.codes.shape == (300, 256) and q.scales.shape == (2, 3) and q.scales.dtype == torch.uint8 and q.rows == 300
    q = lib.empty_quantized_fp8(300, 130, device="cpu")
    assert q.scales.shape == (2, 300) and q.scales.dtype == torch.float32
    assert lib.empty_quantized_fp8(0, 0, device="cpu").codes.shape == (0, 0)


def test_quantize_binding_refusals():
    x = t(32, 200, dtype=torch.bfloat16)
    raises(lambda: lib.quantize_fp8(x), "row or col is required")
    raises(lambda: lib.quantize_fp8(t(32, 200), row=operand(32, 200)), "dtype")
    raises(lambda: lib.quantize_fp8(torch.zeros(32, 200, dtype=torch.bfloat16), row=operand(32, 200)), "device")
    raises(lambda: lib.quantize_fp8(x.t(), row=operand(200, 32)), "unit stride")
    raises(lambda: lib.quantize_fp8(x, row=operand(32, 201)), "expected 32 x 200")
    raises(lambda: lib.quantize_fp8(x, col=operand(32, 200)), "expected 200 x 32")
    raises(lambda: lib.quantize_fp8(x, row=operand(32, 200), col=operand(200, 32, lib.E5M2)), "disagree")
    raises(lambda: lib.quantize_fp8(x, row=operand(32, 200), col=operand(200, 32, e8m0=True)), "disagree")
    raises(lambda: lib.quantize_fp8(x, row=operand(32, 200), col=operand(200, 32, tile=True)), "disagree")
    bad = operand(32, 200)
    bad.scales = t(2, 33)
    raises(lambda: lib.quantize_fp8(x, row=bad), "scales")
    bad = operand(32, 200)
    bad.codes = t(32, 200, dtype=torch.uint8)  # not padded to 256
    raises(lambda: lib.quantize_fp8(x, row=bad), "codes")
    bad = operand(32, 200)
    bad.fmt = 7
    raises(lambda: lib.quantize_fp8(x, row=bad), "unknown format")
    bad = operand(32, 200)
    bad.codes = t(32, 512, dtype=torch.uint8)[:, ::2]
    raises(lambda: lib.quantize_fp8(x, row=bad), "contiguous")
    raises(lambda: lib.quantize_fp8(x, row=(1, 2)), "Fp8Quantized")


@pytest.mark.parametrize("fn", ["gemm_fp8_nt", "gemm_fp8_fprop", "gemm_fp8_dgrad", "gemm_fp8_wgrad"])
def test_gemm_binding_refusals(fn):
    call = getattr(lib, fn)
    a, b, out = operand(32, 200), operand(48, 200), t(32, 48)
    raises(lambda: call(a, operand(48, 201), out), "contraction axis")
    raises(lambda: call(a, operand(48, 200, e8m0=True), out), "different types")
    raises(lambda: call(a, b, t(32, 47)), "output must be")
    raises(lambda: call(a, b, t(32, 48, dtype=torch.float16)), "dtype")
    raises(lambda: call(a, b, t(48, 32).t()), "contiguous")
    raises(lambda: call(a, b, torch.zeros(32, 48)), "device")
    host = operand(32, 200)
    host.scales = torch.zeros(2, 32)
    raises(lambda: call(host, b, out), "device")


def test_dropout_binding_refusals():
    x, o = t(8, 32), t(8, 32)
    for p in (-0.5, 1.5, float("nan")):
        raises(lambda: lib.dropout(x, p, 0, 0, o), "p must lie")
    raises(lambda: lib.dropout(x, 0.5, -1, 0, o), "seed must fit")
    raises(lambda: lib.dropout(x, 0.5, 0, 1 << 32, o), "seed must fit")
    raises(lambda: lib.dropout(x, 0.5, 0, 0, t(8, 33)), "shape")
    raises(lambda: lib.dropout(x, 0.5, 0, 0, t(8, 32, dtype=torch.float16)), "dtype")
    raises(lambda: lib.dropout(x, 0.5, 0, 0, o, residual=t(8, 32, dtype=torch.bfloat16)), "dtype")
    raises(lambda: lib.dropout(x, 0.5, 0, 0, o, residual=t(8, 31)), "shape")
    raises(lambda: lib.dropout(x, 0.5, 0, 0, o, amax=t(2)), "exactly one")
    raises(lambda: lib.dropout(x, 0.5, 0, 0, torch.zeros(8, 32)), "device")
    raises(lambda: lib.dropout_backward(torch.zeros(8, 32), 0.5, 0, 0, o), "device")
    raises(lambda: lib.dropout_backward(x, 2.0, 0, 0, o), "p must lie")


def test_status_text_names_the_call(L):
    e = lib.Ue5m3Fp4Error(ESHAPE, "ue5m3fp4_quantize_fp8")
    assert "ue5m3fp4_quantize_fp8" in str(e) and e.status == ESHAPE
    assert isinstance(L, ctypes.CDLL)
