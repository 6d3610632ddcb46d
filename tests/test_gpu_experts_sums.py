"""GPU tests of the grouped products where their sums are longest.

The bar is the library's, 1e-5 * |ts| * sum |a b|, at every length.  An fp32 sum
of n matrix instructions is off by up to n * 2^-24 of it where all terms are alike
and of one sign: 2^11 instructions (32768 elements of K here) stay near the bar,
2^17 do not, so long sums have to be joined from shorter ones: of 256 instructions,
2^-16 = 1.5e-5 at most, half of that on average over a growing sum.
"""

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as lib
from devhelpers import dev_scalar
from test_gpu_experts_sizes import dev_i32, empty, offsets_of, rand_operand, values

pytestmark = pytest.mark.gpu

KINDS = ["signs", "positive", "equal"]


def long_operand(rows, cols, seed, kind):
    """Random codes and scales; without signs; or one value in all places, so that the sum rounds the same way each time."""
    q = rand_operand(rows, cols, seed)
    if kind == "positive":
        q.codes.bitwise_and_(0x77)
    elif kind == "equal":
        q.codes.fill_(0x55)  # 3
        q.scales.fill_(0x79 + 2 * (seed % 3))
    return q


def sampled(n):
    return sorted({0, n - 1, *np.random.default_rng(n).integers(0, n, 20).tolist()})


def products(u, v):
    """u v^T and |u| |v|^T in fp64, the long axis (a multiple of 16) in 16 pieces side by side."""
    import torch

    u, v = u.view(len(u), 16, -1).transpose(0, 1).contiguous(), v.view(len(v), 16, -1).permute(1, 2, 0).contiguous()
    return torch.bmm(u, v).sum(0), torch.bmm(u.abs(), v.abs()).sum(0)


def dot(a, ia, b, ib, first, n):
    """fp64 products of rows ia of a and ib of b over n columns from `first` on, in slices, and the sums of |a b|."""
    import torch

    ref = torch.zeros((len(ia), len(ib)), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    part = lambda q, i, c, m: values(lib.Quantized(q.codes[i, c // 2:(c + m) // 2], q.scales[i, c // 16:(c + m) // 16], q.ts))  # noqa: E731
    for c in range(first, first + n, 1 << 19):
        m = min(1 << 19, first + n - c)
        r, s = products(part(a, ia, c, m), part(b, ib, c, m))
        ref += r
        bound += s
    return ref, 1e-5 * bound


def check_sampled(out, ia, ib, ref, lim):
    got = out[ia][:, ib].double()
    assert bool(((got - ref).abs() <= lim).all()), float(((got - ref).abs() / (lim / 1e-5)).max())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N", [(40, 24),       # 64 x 64 tiles, waves share the contraction
                                 (2100, 2000),   # tiles of 128 rows
                                 (4112, 2000)])  # of 256 and 16 rows
def test_wgrad_of_an_expert_with_many_rows(cuda_device, M, N, kind):
    rows = 2_100_000
    counts = [3, rows - 203, 200]
    off, P = offsets_of(counts), lib.rows_padded(rows, 3)
    a, b = long_operand(M, P, 1, kind), long_operand(N, P, 2, kind)
    dw = empty((3, M, N), False)
    lib.gemm_grouped_wgrad(a, b, dev_i32(off), dw)
    ia, ib = sampled(M), sampled(N)
    for g, n in enumerate(counts):
        p = 128 * (-(-int(off[g]) // 128) + g)
        check_sampled(dw[g], ia, ib, *dot(a, ia, b, ib, p, -(-n // 128) * 128))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,N,K", [(40, 24, 1 << 21), (70, 100, (1 << 21) + 2064),      # 64 x 64 tiles
                                      (90, 8200, 1 << 18), (21, 33000, (1 << 18) + 2064),  # 128 rows
                                      (1100, 16400, (1 << 18) + 16), (1100, 16400, 1 << 18)])  # 256 rows
def test_grouped_rows_of_long_contractions(cuda_device, rows, N, K, kind):
    import torch

    counts = [rows - 9, 0, 9]
    a, w = long_operand(rows, K, 3, kind), long_operand(3 * N, K, 4, kind)
    w = lib.ExpertWeights(w.codes.view(3, N, -1), w.scales.view(3, N, -1), torch.full((3,), 0.5, device="cuda"))
    y = empty((rows, N), False)
    lib.gemm_grouped_fprop(a, w, dev_i32(offsets_of(counts)), y)
    ib = sampled(N)
    for g, ia in ((0, sampled(rows - 9)), (2, list(range(rows - 9, rows)))):
        check_sampled(y, ia, ib, *dot(a, ia, w.expert(g), ib, 0, K))


@pytest.mark.parametrize("bf16", [False, True])
def test_long_sums_of_infinities_and_nan(cuda_device, bf16):
    """A sum that leaves fp32's range stays infinite, a NaN block stays NaN, and neither reaches other results."""
    import torch

    K, N, rows = 1 << 18, 8200, 66
    a, w = long_operand(rows, K, 5, "equal"), long_operand(N, K, 6, "positive")
    a.scales[1].fill_(0xFE)         # 3 * 114688
    w.codes[7].fill_(0x77)
    w.scales[7].fill_(0xFE)
    w.scales[9, 77] = 0xFF
    a.ts.fill_(3e30)
    y = empty((rows, N), bf16)
    lib.gemm_grouped_fprop(a, lib.ExpertWeights(w.codes[None], w.scales[None], w.ts), dev_i32([0, rows]), y)
    got = y.double()
    assert bool(got[:, 9].isnan().all()) and float(got[1, 7]) == float("inf")
    ib = [j for j in sampled(N) if j not in (7, 9)]
    ref, lim = dot(a, [0, 2, 65], w, ib, 0, K)
    if bf16:
        lim = lim + 2.0 ** -8 * (ref.abs() + lim)
    check_sampled(y, [0, 2, 65], ib, ref, lim)
    assert torch.equal(y.isnan().sum(0) == rows, torch.arange(N, device="cuda") == 9)
