"""Pins of the routed experts' oracle: one expert is the definition for one
matrix, worked layouts, and products by explicit loops in exact arithmetic."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import experts as ox
from oracle import formats, gemm, quantize
from workloads import random_bf16


def test_worked_layout():
    # rows 3 .. 7, none, 8 .. 136, 137: columns from 128 (1 + 0), 128 (1 + 1), 128 (1 + 2), 128 (2 + 3)
    assert ox.spans([3, 8, 8, 137, 138]) == [(3, 5, 128, 128), (8, 0, 256, 0), (8, 129, 384, 256), (137, 1, 640, 128)]
    assert ox.rows_padded(138, 4) == 128 * 6 and ox.rows_padded(0, 2) == 256


def test_one_expert_is_one_matrix():
    bits = random_bf16((256, 32), 1, "gradient")
    for rounding in (0, 1):
        r = ox.quantize_row(bits, [0, 256], np.float32(1e-3), rounding, 9, 4)
        want = quantize.quantize_blockscale(bits, np.float32(1e-3), rounding, 9, 4, 0)
        assert r[2].all() and np.array_equal(r[0], want[0]) and np.array_equal(r[1], want[1])
    codes, scales, written = ox.quantize_col(bits, [0, 256], np.float32(1e-3))
    want = quantize.quantize_blockscale(bits, np.float32(1e-3), orientation=1)
    assert np.array_equal(codes[:, :128], want[0]) and np.array_equal(scales[:, :16], want[1])
    assert written[:16].all() and not written[16:].any()


@pytest.mark.parametrize("counts", [[5, 0, 130, 1], [128, 16]])
def test_transposed_blocks_hold_one_expert(counts):
    off = np.concatenate([[0], np.cumsum(counts)])
    bits = random_bf16((int(off[-1]), 16), 2)
    codes, scales, written = ox.quantize_col(bits, off, np.float32(0.01))
    for b, n, p, wide in ox.spans(off):
        alone = np.zeros((wide, 16), dtype=np.uint16)
        alone[:n] = bits[b:b + n]
        if n == 0:
            continue
        want = quantize.quantize_blockscale(alone, np.float32(0.01), orientation=1)
        assert np.array_equal(codes[:, p // 2:(p + wide) // 2], want[0])
        assert np.array_equal(scales[:, p // 16:(p + wide) // 16], want[1])
        assert written[p // 16:(p + wide) // 16].all()
    assert written.sum() == sum(-(-n // 128) * 8 for n in counts)


def test_gather_and_amax():
    bits = np.array([[0x3F80] * 16, [0xC000] * 16, [0x7F80] * 16], dtype=np.uint16)  # 1, -2, inf
    got = ox.gather(bits, [1, -1, 0, 3, 1])
    assert np.array_equal(got, np.stack([bits[1], 0 * bits[0], bits[0], 0 * bits[0], bits[1]]))
    assert ox.amax(bits, [0, 1, 2]) == 2.0 and np.isinf(ox.amax(bits, [2, 3]))


def exact_values(codes, scales):
    """Fractions, element by element."""
    rows, cols = codes.shape[0], codes.shape[1] * 2
    e2m1 = [Fraction(v) for v in (0, 0.5, 1, 1.5, 2, 3, 4, 6)]
    out = []
    for i in range(rows):
        line = []
        for k in range(cols):
            c = (int(codes[i, k // 2]) >> (4 * (k % 2))) & 15
            s = int(scales[i, k // 16])
            e, f = s >> 3, s & 7
            scale = Fraction(f, 8) * Fraction(1, 2 ** 14) if e == 0 else (1 + Fraction(f, 8)) * Fraction(2) ** (e - 15)
            line.append(e2m1[c & 7] * scale * (-1 if c & 8 else 1))
        out.append(line)
    return out


def test_products_by_exact_loops():
    rng = np.random.default_rng(3)
    op = lambda r, c: (rng.integers(0, 256, (r, c // 2)).astype(np.uint8),  # noqa: E731
                       rng.integers(0x60, 0x90, (r, c // 16)).astype(np.uint8))
    off, E, rows, N, K = [1, 3, 3, 5], 3, 6, 3, 32
    a, w = op(rows, K), [op(N, K) for _ in range(E)]
    wc, ws = np.stack([q[0] for q in w]), np.stack([q[1] for q in w])
    ts = [0.5, 2.0, 0.25]
    c, bound, owned = ox.gemm_rows(a, 4.0, wc, ws, ts, off)
    assert owned.tolist() == [False, True, True, True, True, False]
    av = exact_values(*a)
    x = random_bf16((rows, K), 4)
    xv = [[Fraction(float(v)) for v in line] for line in formats.bf16_to_f32(x)]
    wo, _, _ = ox.weight_only(x, wc, ws, ts, off)
    for g, (b, n, _, _) in enumerate(ox.spans(off)):
        wv = exact_values(*w[g])
        for i in range(b, b + n):
            for j in range(N):
                terms = [p * q for p, q in zip(av[i], wv[j])]
                assert c[i, j] == float(sum(terms) * Fraction(4) * Fraction(ts[g]))
                assert bound[i, j] == pytest.approx(float(sum(map(abs, terms)) * Fraction(4) * Fraction(ts[g])), rel=1e-12)
                want = sum(p * q for p, q in zip(xv[i], wv[j])) * Fraction(ts[g])
                assert wo[i, j] == pytest.approx(float(want), rel=1e-12, abs=1e-30)
    P = ox.rows_padded(rows, E)
    at, bt = op(2, P), op(3, P)
    dw, _ = ox.gemm_wgrad(at, 1.0, bt, 0.5, off)
    assert dw.shape == (E, 2, 3) and (dw[1] == 0).all()
    for g, (_, _, p, n) in enumerate(ox.spans(off)):
        part = [(q[0][:, p // 2:(p + n) // 2], q[1][:, p // 16:(p + n) // 16]) for q in (at, bt)]
        if n:
            u, v = exact_values(*part[0]), exact_values(*part[1])
            for i in range(2):
                for j in range(3):
                    assert dw[g, i, j] == float(sum(p_ * q_ for p_, q_ in zip(u[i], v[j])) * Fraction(1, 2))
    assert gemm.gemm_nt(*part[0], 1.0, *part[1], 0.5)[0].shape == (2, 3)
