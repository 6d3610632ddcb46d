"""CPU tests of libue5m3fp4_experts' refusals: the C ABI rejects bad arguments
on the host before any HIP call (the pointers are never dereferenced), and the
Python binding rejects malformed operands before it takes a pointer.  The
arithmetic that keeps kernels inside their operands whatever the offsets hold
is checked here too, in a model of it."""

import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import fp4_block_scaled_amax_amd as lib
from oracle import experts as ox
from test_binding_checks import Dev, raises

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ue5m3fp4_experts.h")
OK, EINVAL, ESHAPE, EALIGN, ERANGE = 0, -1, -2, -3, -5
P = 0x10000


@pytest.fixture(scope="module")
def L():
    return lib.load_experts_library()


def test_exports_and_c99_header(L, tmp_path):
    names = sorted(re.findall(r"UE5M3FP4_API\s+int\s+(ue5m3fp4_\w+)\(", open(HEADER).read()))
    out = subprocess.run(["nm", "-D", "--defined-only", lib.EXPERTS_LIB_PATH], capture_output=True, text=True).stdout
    assert sorted(re.findall(r" T (\S+)", out)) == names and len(names) == 4
    gcc = shutil.which("gcc")
    if gcc:
        src = tmp_path / "a.c"
        src.write_text('#include "ue5m3fp4_layer.h"\n#include "ue5m3fp4_experts.h"\nint main(void) { return UE5M3FP4_OUT_BF16; }\n')
        subprocess.run([gcc, "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-c", str(src), "-o", str(tmp_path / "a.o")], check=True)


def qg(L, x=P, xr=32, cols=32, ld=32, idx=None, rows=32, off=P, E=2, ts=P, rnd=0, rc=P, rs=P, cc=2 * P, cs=2 * P, am=None):
    return L.ue5m3fp4_quantize_grouped(x, xr, cols, ld, idx, rows, off, E, ts, rnd, 0, 0, rc, rs, cc, cs, am, None)


def test_quantize_argument_checks(L):
    assert qg(L, rows=-1, xr=-1) == EINVAL and qg(L, E=-1) == EINVAL and qg(L, rnd=2) == EINVAL
    assert qg(L, x=None) == EINVAL and qg(L, off=None) == EINVAL and qg(L, ts=None) == EINVAL
    assert qg(L, rc=None) == EINVAL and qg(L, cs=None) == EINVAL
    assert qg(L, rc=None, rs=None, cc=None, cs=None) == EINVAL
    assert qg(L, cc=P) == EINVAL and qg(L, cs=P) == EINVAL  # one buffer for both outputs
    assert qg(L, xr=31) == ESHAPE and qg(L, cols=40, ld=40) == ESHAPE and qg(L, ld=24) == ESHAPE
    assert qg(L, ld=36) == EALIGN and qg(L, x=P + 8) == EALIGN and qg(L, rc=P + 8) == EALIGN and qg(L, cs=2 * P + 4) == EALIGN
    assert qg(L, off=P + 2) == EALIGN and qg(L, ts=P + 2) == EALIGN and qg(L, idx=P + 2) == EALIGN and qg(L, am=P + 1) == EALIGN
    assert qg(L, rows=1 << 31, idx=P) == ERANGE and qg(L, E=65537) == ERANGE and qg(L, ld=1 << 39) == ERANGE
    assert qg(L, xr=(1 << 31) - 1, rows=(1 << 31) - 1, ld=1 << 62) == ERANGE
    assert qg(L, rows=(1 << 31) - 128, xr=(1 << 31) - 128, E=2) == ERANGE  # rows_padded = 2^31 + 128
    assert qg(L, cols=1 << 20, ld=1 << 20, rows=1 << 20, xr=1, idx=P) == ERANGE  # cols * rows_padded
    assert qg(L, rows=0, xr=0, x=None) == OK and qg(L, cols=0, ld=0, x=None) == OK and qg(L, E=0, off=None) == OK


def gr(L, ac=P, as_=P, at=P, bc=P, bs=P, bt=P, n=1, off=P, E=2, rows=32, N=32, K=32, c=P, ct=0, am=None):
    return L.ue5m3fp4_gemm_grouped_nt(ac, as_, at, bc, bs, bt, n, off, E, rows, N, K, c, ct, am, None)


def test_gemm_argument_checks(L):
    assert gr(L, E=-1) == EINVAL and gr(L, rows=-1) == EINVAL and gr(L, N=-1) == EINVAL and gr(L, K=-16) == EINVAL
    assert gr(L, ct=2) == EINVAL and gr(L, n=3) == EINVAL and gr(L, n=0) == EINVAL and gr(L, ct=1, am=P) == EINVAL
    for name in ("ac", "as_", "at", "bc", "bs", "bt", "off", "c"):
        assert gr(L, **{name: None}) == EINVAL
        assert gr(L, **{name: P + 2}, K=128) == EALIGN
    assert gr(L, bc=P + 4) == EALIGN and gr(L, bs=P + 4, K=256) == EALIGN and gr(L, as_=P + 8) == EALIGN
    assert gr(L, am=P + 2) == EALIGN and gr(L, c=P + 4) == EALIGN
    assert gr(L, K=40) == ESHAPE
    assert gr(L, rows=1 << 31) == ERANGE and gr(L, N=1 << 31) == ERANGE and gr(L, K=1 << 24) == ERANGE
    assert gr(L, rows=1 << 20, N=1 << 20) == ERANGE and gr(L, E=65536, N=1 << 12, K=1 << 12) == ERANGE
    assert gr(L, E=65537) == ERANGE
    assert gr(L, E=0, n=0, off=None) == OK and gr(L, rows=0, c=None) == OK and gr(L, N=0, c=None) == OK


def gw(L, ac=P, as_=P, at=P, bc=P, bs=P, bt=P, off=P, E=2, rows=32, M=32, N=32, c=P, ct=0):
    return L.ue5m3fp4_gemm_grouped_wgrad(ac, as_, at, bc, bs, bt, off, E, rows, M, N, c, ct, None)


def test_wgrad_argument_checks(L):
    assert gw(L, E=-1) == EINVAL and gw(L, rows=-1) == EINVAL and gw(L, M=-1) == EINVAL and gw(L, N=-1) == EINVAL
    assert gw(L, ct=2) == EINVAL
    for name in ("ac", "as_", "at", "bc", "bs", "bt", "off", "c"):
        assert gw(L, **{name: None}) == EINVAL
        assert gw(L, **{name: P + 2}) == EALIGN
    assert gw(L, rows=(1 << 24) - 256) == ERANGE and gw(L, M=1 << 31) == ERANGE and gw(L, E=65537) == ERANGE
    assert gw(L, rows=1 << 20, M=1 << 20) == ERANGE and gw(L, E=65536, M=1 << 12, N=1 << 12) == ERANGE
    assert gw(L, E=0, off=None) == OK and gw(L, M=0) == OK and gw(L, N=0) == OK


def wo(L, x=P, ldx=32, wc=P, ws=P, wt=P, n=1, off=P, E=2, rows=4, N=32, K=32, out=P, ot=0, ldo=32):
    return L.ue5m3fp4_gemm_weight_only(x, ldx, wc, ws, wt, n, off, E, rows, N, K, out, ot, ldo, None)


def test_weight_only_argument_checks(L):
    assert wo(L, rows=-1) == EINVAL and wo(L, ldx=-8) == EINVAL and wo(L, ldo=-1) == EINVAL and wo(L, ot=2) == EINVAL
    assert wo(L, off=None) == EINVAL                # several experts need offsets
    assert wo(L, n=3) == EINVAL and wo(L, n=0) == EINVAL
    for name in ("x", "wc", "ws", "wt", "out"):
        assert wo(L, **{name: None}) == EINVAL
        assert name == "ws" or wo(L, **{name: P + 2}) == EALIGN
    assert wo(L, wc=P + 4) == EALIGN and wo(L, x=P + 8) == EALIGN and wo(L, out=P + 8) == EALIGN
    assert wo(L, off=P + 2) == EALIGN and wo(L, ldx=36) == EALIGN
    assert wo(L, K=40, ldx=40) == ESHAPE and wo(L, ldx=24) == ESHAPE and wo(L, ldo=31) == ESHAPE
    assert wo(L, rows=1 << 31) == ERANGE and wo(L, K=1 << 24, ldx=1 << 24) == ERANGE and wo(L, ldx=1 << 39) == ERANGE and wo(L, ldo=1 << 39) == ERANGE
    assert wo(L, E=65536, N=1 << 12, K=1 << 12) == ERANGE and wo(L, E=65537) == ERANGE
    assert wo(L, rows=0, out=None) == OK and wo(L, N=0, ldo=0) == OK and wo(L, E=0, n=0, off=None) == OK


# ------------------------------------------------------------------- binding --

def dev(*shape, dtype=torch.float32):
    return Dev(torch.zeros(shape, dtype=dtype))


u8 = torch.uint8


def quantized(rows, cols):
    return lib.Quantized(dev(rows, cols // 2, dtype=u8), dev(rows, cols // 16, dtype=u8), dev(1))


def weights(E, R, C, ts=1):
    return lib.ExpertWeights(dev(E, R, C // 2, dtype=u8), dev(E, R, C // 16, dtype=u8), dev(ts))


def offs(E):
    return dev(E + 1, dtype=torch.int32)


def test_shapes_and_views():
    w = lib.empty_expert_weights(3, 10, 32, torch.ones(3))
    assert w.experts == 3 and w.codes.shape == (3, 10, 16) and w.scales.shape == (3, 10, 2)
    q = w.expert(1)
    assert q.rows == 10 and q.cols == 32 and q.ts.numel() == 1 and q.ts.data_ptr() == w.ts[1:].data_ptr()
    assert lib.empty_expert_weights(3, 10, 32, torch.ones(1)).expert(2).ts.numel() == 1
    assert lib.rows_padded(0, 4) == 512 and lib.rows_padded(1, 1) == 256 and lib.rows_padded(128, 2) == 384


def test_quantize_binding_refusals():
    x, o, ts = dev(32, 64, dtype=torch.bfloat16), offs(2), dev(1)
    call = lib.quantize_grouped
    raises(lambda: call(x, o, ts), "row, col or amax")
    raises(lambda: call(x, o, None, row=quantized(32, 64)), "tensor_scale is required")
    raises(lambda: call(dev(32, 64), o, ts, row=quantized(32, 64)), "dtype")
    raises(lambda: call(x, dev(3), ts, row=quantized(32, 64)), "dtype")
    raises(lambda: call(x, dev(0, dtype=torch.int32), ts, row=quantized(32, 64)), "experts")
    raises(lambda: call(x, torch.zeros(3, dtype=torch.int32), ts, row=quantized(32, 64)), "device")
    raises(lambda: call(x.t(), o, ts, row=quantized(64, 32)), "unit stride")
    raises(lambda: call(x, o, ts, row=quantized(31, 64)), "do not match")
    raises(lambda: call(x, o, ts, col=quantized(64, 32)), "do not match")       # 384 columns: rows_padded(32, 2)
    raises(lambda: call(x, o, ts, row=quantized(32, 64), index=dev(40, dtype=torch.int32)), "do not match")
    raises(lambda: call(x, o, ts, row=quantized(40, 64), index=dev(40, dtype=torch.int64)), "dtype")
    raises(lambda: call(x, o, dev(2), row=quantized(32, 64)), "exactly one")
    raises(lambda: call(x, o, ts, row=quantized(32, 64), amax=dev(2)), "exactly one")
    raises(lambda: call(x, o, ts, row=quantized(32, 64), seed=-1), "seed must fit")
    raises(lambda: call(x, o, ts, row=quantized(32, 64), offset=1 << 32), "seed must fit")


@pytest.mark.parametrize("fn", ["gemm_grouped_fprop", "gemm_grouped_dgrad"])
def test_gemm_binding_refusals(fn):
    call = getattr(lib, fn)
    a, w, o, out = quantized(32, 64), weights(2, 48, 64), offs(2), dev(32, 48)
    raises(lambda: call(a, w, offs(3), out), "experts")
    raises(lambda: call(a, weights(2, 48, 80), o, out), "contraction axis")
    raises(lambda: call(a, weights(2, 48, 64, ts=3), o, out), "one per expert")
    raises(lambda: call(a, quantized(48, 64), o, out), "ExpertWeights")
    raises(lambda: call(w, w, o, out), "Quantized operand")
    raises(lambda: call(a, w, o, dev(32, 47)), "must be a contiguous")
    raises(lambda: call(a, w, o, dev(48, 32).t()), "contiguous")
    raises(lambda: call(a, w, o, dev(32, 48, dtype=torch.float16)), "dtype")
    raises(lambda: call(a, w, o, out, amax=dev(1)), "bf16 outputs")
    raises(lambda: call(a, w, o, torch.zeros(32, 48)), "device")
    bad = weights(2, 48, 64)
    bad.scales = dev(2, 48, 5, dtype=u8)
    raises(lambda: call(a, bad, o, out), "do not match")


def test_wgrad_binding_refusals():
    o, dw = offs(2), dev(2, 48, 64)
    raises(lambda: lib.gemm_grouped_wgrad(quantized(48, 368), quantized(64, 368), o, dw), "rows_padded")
    raises(lambda: lib.gemm_grouped_wgrad(quantized(48, 128), quantized(64, 128), o, dw), "rows_padded")
    raises(lambda: lib.gemm_grouped_wgrad(quantized(48, 384), quantized(64, 512), o, dw), "rows_padded")
    raises(lambda: lib.gemm_grouped_wgrad(quantized(48, 384), quantized(64, 384), o, dev(2, 64, 48)), "must be a contiguous")
    raises(lambda: lib.gemm_grouped_wgrad(quantized(48, 384), quantized(64, 384), o, dev(1, 48, 64)), "must be a contiguous")


def test_weight_only_binding_refusals():
    x, out, o = dev(4, 64, dtype=torch.bfloat16), dev(4, 48), offs(2)
    call = lib.gemm_weight_only
    raises(lambda: call(x, weights(2, 48, 64), out), "Quantized operand")
    raises(lambda: call(x, quantized(48, 64), out, offsets=o), "ExpertWeights")
    raises(lambda: call(x, weights(3, 48, 64), out, offsets=o), "experts")
    raises(lambda: call(x, quantized(48, 80), out), "contraction axis")
    raises(lambda: call(dev(4, 64), quantized(48, 64), out), "dtype")
    raises(lambda: call(x, quantized(48, 64), dev(4, 47)), "must be a")
    raises(lambda: call(x, quantized(48, 64), dev(48, 4).t()), "unit stride")
    raises(lambda: call(x, quantized(48, 64), dev(4, 48, dtype=torch.float16)), "dtype")
    raises(lambda: call(torch.zeros(4, 64, dtype=torch.bfloat16), quantized(48, 64), out), "device")


# ------------------------------------------------------------------- offsets --

def test_any_offsets_stay_inside_the_operands():
    """The kernels' clamped view of offsets (begin in [0, rows], end in [begin, rows]): every group's rows and its
    columns in the transposed operand lie inside, and ordered offsets give disjoint columns."""
    rng = np.random.default_rng(0)
    for _ in range(2000):
        rows, E = int(rng.integers(0, 600)), int(rng.integers(1, 9))
        raw = rng.integers(-1000, 2000, E + 1) if rng.random() < 0.5 else np.sort(rng.integers(0, rows + 1, E + 1))
        padded, last = lib.rows_padded(rows, E), 0
        ordered = bool((np.diff(raw) >= 0).all() and raw[0] >= 0 and raw[-1] <= rows)
        for g in range(E):
            begin = min(max(int(raw[g]), 0), rows)
            end = min(max(int(raw[g + 1]), begin), rows)
            first = 128 * (-(-begin // 128) + g)
            assert 0 <= begin <= end <= rows and first + -(-(end - begin) // 128) * 128 <= padded
            if ordered:
                assert first >= last
                last = first + -(-(end - begin) // 128) * 128
        if ordered:
            assert [(b, p) for b, _, p, _ in ox.spans(raw)] == [(int(raw[g]), 128 * (-(-int(raw[g]) // 128) + g)) for g in range(E)]
            full = sum((n + 127) // 256 for _, n, _, _ in ox.spans(raw))
            rest = sum(n > 256 * ((n + 127) // 256) for _, n, _, _ in ox.spans(raw))
            assert full + rest <= rows // 256 + min(E, rows)  # the grid of the grouped products
