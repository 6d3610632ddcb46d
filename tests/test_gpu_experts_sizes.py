"""GPU tests of the routed experts' operators where their kernels change shape or
their offsets grow: tall tiles and every rest behind them, every variant of the
weight-only product, operands and results past 2^32 bytes, and offsets that are no
offsets.

Operands are random codes and scale bytes; the definition is fp64 products of
their values (decoded by the oracle's tables) on the device.  The bar is
the library's: 1e-5 * |ts| * sum |a b|, bf16 half a step (2^-8) further.
"""

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as lib
from devhelpers import dev_bf16, dev_scalar
from oracle import formats
from workloads import random_bf16

pytestmark = pytest.mark.gpu


def gen(seed):
    import torch

    return torch.Generator("cuda").manual_seed(seed)


def rand_operand(rows, cols, seed, ts=1.0):
    """Random codes; scales of 2^-4 to 2 (bytes 0x58 .. 0x7F), some of them 0."""
    import torch

    g = gen(seed)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(0x57, 0x80, (rows, cols // 16), dtype=torch.uint8, device="cuda", generator=g)
    scales[scales == 0x57] = 0
    return lib.Quantized(codes, scales, dev_scalar(ts))


def rand_weights(experts, rows, cols, seed, one_ts=False):
    import torch

    q = rand_operand(experts * rows, cols, seed)
    ts = torch.full((1,), 0.75, device="cuda") if one_ts else 0.5 + torch.rand(experts, device="cuda", generator=gen(seed + 1))
    return lib.ExpertWeights(q.codes.view(experts, rows, -1), q.scales.view(experts, rows, -1), ts)


def values(q):
    """fp64 values of an operand, its tensor scale included."""
    import torch

    e2m1 = torch.tensor(formats.e2m1_decode(np.arange(16, dtype=np.uint8)), dtype=torch.float64, device="cuda")
    ue5m3 = torch.tensor(formats.ue5m3_decode(np.arange(256, dtype=np.uint8)), dtype=torch.float64, device="cuda")
    c = q.codes.long()
    v = torch.stack([e2m1[c & 15], e2m1[c >> 4]], dim=-1).flatten(-2)
    return v * ue5m3[q.scales.long()].repeat_interleave(16, dim=-1) * q.ts.double()


def offsets_of(counts, before=0):
    return np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int64)


def dev_i32(v):
    import torch

    return torch.tensor([int(i) for i in v], dtype=torch.int32, device="cuda")


def empty(shape, bf16):
    import torch

    return torch.full(shape, -77.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")


def check(out, a, b, bf16):
    """Rows of out against a b^T."""
    ref, bound = a @ b.t(), 1e-5 * (a.abs() @ b.abs().t())
    if bf16:
        bound = bound + 2.0 ** -8 * (ref.abs() + bound)
    assert bool(((out.double() - ref).abs() <= bound).all())


# --------------------------------------------------------------- tall tiles --

# Tiles of 256 rows (N 8200), of 128 (N 700) and of 64 with split contractions (N 100).
# Behind full tiles: rests of 1 .. 32, 33 .. 64, 65 .. 128 and 129 .. 255, and none
TALL = [256, 1, 33, 65, 129, 257, 300, 384, 385, 0, 511, 512, 192, 193, 440]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,K", [(8200, 128), (8197, 384), (8200, 272), (704, 128), (701, 1040), (720, 400), (704, 16), (704, 48),
                                 (100, 1024), (101, 1104), (130, 528), (64, 32)])
def test_grouped_rows_in_many_tiles(cuda_device, N, K, bf16):
    counts, before, behind = TALL, 3, 5
    off, E = offsets_of(counts, before), len(counts)
    rows = int(off[-1]) + behind
    a, w = rand_operand(rows, K, 1, 0.5), rand_weights(E, N, K, 2)
    y, amax = empty((rows, N), bf16), dev_scalar(0.0)
    lib.gemm_grouped_fprop(a, w, dev_i32(off), y, amax=amax if bf16 else None)
    av = values(a)
    for g in range(E):
        check(y[off[g]:off[g + 1]], av[off[g]:off[g + 1]], values(w.expert(g)), bf16)
    assert bool((y[:before] == -77.0).all()) and bool((y[off[-1]:] == -77.0).all())
    if bf16:
        assert float(amax) == float(y[before:off[-1]].float().abs().max())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N", [(2100, 5000), (2050, 5104), (1801, 6001), (2100, 1500), (700, 701), (720, 704), (130, 68), (33, 67)])
def test_wgrad_in_many_tiles(cuda_device, M, N, bf16):
    counts = [0, 1, 300, 128, 1165]
    off, E = offsets_of(counts, 2), len(counts)
    rows = int(off[-1]) + 1
    P = lib.rows_padded(rows, E)
    a, b = rand_operand(M, P, 3, 0.5), rand_operand(N, P, 4)
    dw = empty((E, M, N), bf16)
    lib.gemm_grouped_wgrad(a, b, dev_i32(off), dw)
    for g in range(E):
        p, n = 128 * (-(-int(off[g]) // 128) + g), -(-counts[g] // 128) * 128
        part = [values(lib.Quantized(q.codes[:, p // 2:(p + n) // 2], q.scales[:, p // 16:(p + n) // 16], q.ts)) for q in (a, b)]
        check(dw[g], part[0], part[1], bf16)
    assert bool((dw[0] == 0).all())


# ---------------------------------------------------- the weight-only product --

@pytest.mark.parametrize("K", [16, 512, 528, 1152, 4224, 5648])
@pytest.mark.parametrize("rows,N", [(1, 16), (1, 8209), (1, 32790), (2, 16389), (4, 700), (9, 8195), (16, 16400), (16, 330), (31, 16390),
                                    (32, 330), (33, 8195), (64, 650), (65, 650), (200, 4099), (20, 8200), (20, 65540), (40, 65540),
                                    (3, 32777), (9, 32777)])
def test_weight_only_variants(cuda_device, rows, N, K):
    import torch

    bits = random_bf16((rows, K), 7)
    x, q = dev_bf16(bits), rand_operand(N, K, 8, 0.5)
    xv, qv = torch.from_numpy(formats.bf16_to_f32(bits).astype(np.float64)).cuda(), values(q)
    for bf16 in (False, True):
        out = empty((rows, N), bf16)
        lib.gemm_weight_only(x, q, out)
        check(out, xv, qv, bf16)


@pytest.mark.parametrize("K", [512, 400, 1040])
@pytest.mark.parametrize("counts,N", [
    ([1, 0, 0, 0, 0, 0, 1, 0], 1100),               # one token each
    ([1, 0, 0, 0, 0, 0, 1, 0] * 8, 2100),
    ([3, 0, 4, 1, 2, 5] * 12, 260),                 # more experts than lanes of a wave, 1 more than is prepared for
    ([16, 1, 0, 9, 40] * 16, 330),                  # two row blocks of some
    ([33, 0, 31, 10] * 9, 460),
    ([64, 65, 129, 2] * 5, 900),
])
def test_weight_only_variants_of_experts(cuda_device, counts, N, K):
    import torch

    off, E = offsets_of(counts, 1), len(counts)
    rows = int(off[-1]) + 2
    x = torch.randn((rows, K + 8), device="cuda", generator=gen(1)).bfloat16()[:, 8:]
    w = rand_weights(E, N, K, 9, one_ts=K == 400)
    for bf16 in (False, True):
        out = empty((rows, N + 3), bf16)
        lib.gemm_weight_only(x, w, out[:, :N], offsets=dev_i32(off))
        for g in range(E):
            check(out[off[g]:off[g + 1], :N], x[off[g]:off[g + 1]].double(), values(w.expert(g)), bf16)
        assert bool((out[:, N:] == -77.0).all()) and bool((out[0] == -77.0).all()) and bool((out[off[-1]:] == -77.0).all())


@pytest.mark.parametrize("rows", [1, 2, 16, 32, 64])
def test_weight_only_largest_tokens(cuda_device, rows):
    """bf16's largest elements times small weights: no product or partial sum of the definition overflows fp32, so no
    result does.  One nonzero block per row of W at the scale 2^-17, and codes 6: 16 * 6 * 2^-17 * max."""
    import torch

    K, N = 1024, 40
    x = torch.full((rows, K), 3.3895313892515355e38, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((N, K // 2), 0x77, dtype=torch.uint8, device="cuda")
    scales = torch.zeros((N, K // 16), dtype=torch.uint8, device="cuda")
    scales[:, 5] = 1
    q = lib.Quantized(codes, scales, dev_scalar(1.0))
    out = empty((rows, N), False)
    lib.gemm_weight_only(x, q, out)
    check(out, x.double(), values(q), False)


@pytest.mark.parametrize("N,K", [(37, 144), (45, 528), (1305, 2064), (35, 256)])
def test_some_experts_of_a_larger_operand(cuda_device, N, K):
    """Weights that begin at an expert of an operand whose scales have odd sizes: 8-byte aligned codes, scales anywhere."""
    import torch

    w = rand_weights(6, N, K, 30)
    counts = [5, 130, 0, 66]
    off, rows = dev_i32(offsets_of(counts)), sum(counts)
    part = lib.ExpertWeights(w.codes[1:5], w.scales[1:5], w.ts[1:5])
    alone = lib.ExpertWeights(part.codes.clone(), part.scales.clone(), part.ts.clone())
    assert K == 256 or w.scales[1].data_ptr() % 16
    a, x = rand_operand(rows, K, 31), torch.randn((rows, K), device="cuda", generator=gen(32)).bfloat16()
    got, want = empty((rows, N), False), empty((rows, N), False)
    lib.gemm_grouped_fprop(a, part, off, got)
    lib.gemm_grouped_fprop(a, alone, off, want)
    assert torch.equal(got, want)
    check(got[5:135], values(a)[5:135], values(part.expert(1)), False)
    lib.gemm_weight_only(x, part, got, offsets=off)
    lib.gemm_weight_only(x, alone, want, offsets=off)
    assert torch.equal(got, want)
    for tokens in (1, 3, 16, 40):
        y = empty((tokens, N), False)
        lib.gemm_weight_only(x[:tokens], w.expert(3), y)
        check(y, x[:tokens].double(), values(w.expert(3)), False)


# ------------------------------------------------------------ large operands --

def test_quantize_past_32_bit_offsets(cuda_device):
    """2^32 elements: the last expert's rows, in both operands, are those of its rows alone."""
    import torch

    cols, tail = 4112, 300
    rows = (1 << 32) // cols + 1000
    off = [5, 1 << 19, rows - tail - 1, rows - 1]
    block = torch.randn((4093, cols), device="cuda", generator=gen(3)).bfloat16()
    x = block.repeat(-(-rows // 4093), 1)[:rows].contiguous()
    assert x.numel() > 1 << 32
    P, ts = lib.rows_padded(rows, 3), dev_scalar(0.01)
    q = lib.Quantized(*(torch.zeros((rows, cols // n), dtype=torch.uint8, device="cuda") for n in (2, 16)), ts)
    t = lib.Quantized(*(torch.zeros((cols, P // n), dtype=torch.uint8, device="cuda") for n in (2, 16)), ts)
    lib.quantize_grouped(x, dev_i32(off), ts, row=q, col=t)
    first, last = x[off[2]:off[3]].contiguous(), 128 * (-(-off[2] // 128) + 2)
    r1 = lib.empty_quantized(tail, cols, ts)
    padded = torch.zeros((384, cols), dtype=torch.bfloat16, device="cuda")
    padded[:tail] = first
    c1 = lib.empty_quantized(cols, 384, ts)
    lib.quantize_blockscale(first, ts, row=r1)
    lib.quantize_blockscale(padded, ts, col=c1)
    assert torch.equal(q.codes[off[2]:off[3]], r1.codes) and torch.equal(q.scales[off[2]:off[3]], r1.scales)
    assert torch.equal(t.codes[:, last // 2:(last + 384) // 2], c1.codes)
    assert torch.equal(t.scales[:, last // 16:(last + 384) // 16], c1.scales)
    assert bool((q.codes[:5] == 0).all()) and bool((q.codes[rows - 1] == 0).all())
    # the same rows through an index, whose products with the row stride pass 32 bits
    index = torch.arange(off[2], off[3], dtype=torch.int32, device="cuda")
    r2 = lib.empty_quantized(tail, cols, ts)
    lib.quantize_grouped(x, dev_i32([0, tail]), ts, row=r2, index=index)
    assert torch.equal(r2.codes, r1.codes) and torch.equal(r2.scales, r1.scales)


@pytest.mark.parametrize("rows,N,K", [((1 << 20) + 300, 4104, 128),   # C past 2^32 elements
                                      ((1 << 20) + 300, 24, 8320)])   # A past 2^32 bytes
def test_grouped_rows_past_32_bit_offsets(cuda_device, rows, N, K):
    import torch

    off = [0, 77, rows - 299, rows - 1]
    a, w = rand_operand(rows, K, 5), rand_weights(3, N, K, 6)
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    lib.gemm_grouped_fprop(a, w, dev_i32(off), y)
    tail = lib.Quantized(a.codes[off[2]:off[3]], a.scales[off[2]:off[3]], a.ts)
    check(y[off[2]:off[3]], values(tail), values(w.expert(2)), True)


def test_wgrad_past_32_bit_offsets(cuda_device):
    rows, M, N = 2_100_000, 4112, 24
    off = [0, 3, rows - 200, rows]
    P = lib.rows_padded(rows, 3)
    a, b = rand_operand(M, P, 7), rand_operand(N, P, 8)
    assert a.codes.numel() > 1 << 32
    dw = empty((3, M, N), False)
    lib.gemm_grouped_wgrad(a, b, dev_i32(off), dw)
    for g, n in ((0, 128), (2, 256)):
        p = 128 * (-(-off[g] // 128) + g)
        check(dw[g], *(values(lib.Quantized(q.codes[:, p // 2:(p + n) // 2], q.scales[:, p // 16:(p + n) // 16], q.ts))
                       for q in (a, b)), False)


@pytest.mark.parametrize("counts", [[0] * 69 + [1], [0] * 68 + [2, 1], [0] * 69 + [40]])
def test_weight_only_past_32_bit_offsets(cuda_device, counts):
    """70 experts' weights of more than 2^32 bytes: the last expert's product."""
    import torch

    N, K, E, rows = 8192, 16384, 70, sum(counts)
    w = rand_weights(E, N, K, 10)
    assert w.codes.numel() > 1 << 32
    x = torch.randn((rows, K), device="cuda", generator=gen(2)).bfloat16()
    out = empty((rows, N), False)
    lib.gemm_weight_only(x, w, out, offsets=dev_i32(offsets_of(counts)))
    check(out[-counts[-1]:], x[-counts[-1]:].double(), values(w.expert(E - 1)), False)


# ------------------------------------------------- offsets that are no offsets --

@pytest.mark.parametrize("off", [[-5, 10, 40, 200], [40, 30, 20, 10], [0, 1000, 0, 1000], [2 ** 31 - 1, 0, -2 ** 31, 70],
                                 [0, 70, 70, 2 ** 31 - 1], [-1, -1, -1, -1]])
def test_any_offsets_write_inside_the_outputs(cuda_device, off):
    """The kernels clamp what they read: around the outputs nothing changes, whatever the offsets hold."""
    import torch

    rows, K, N, E = 70, 272, 48, 3
    o, P = dev_i32(off), lib.rows_padded(70, 3)

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        pad = 4096 // torch.empty(0, dtype=dtype).element_size()
        whole = torch.full((n + 2 * pad,), 77, dtype=dtype, device="cuda")
        return whole, whole[pad:pad + n].view(shape), pad

    ts = dev_scalar(0.1)
    bufs = [guarded(s, torch.uint8) for s in ((rows, K // 2), (rows, K // 16), (K, P // 2), (K, P // 16))]
    x = torch.randn((rows, K), device="cuda", generator=gen(4)).bfloat16()
    index = dev_i32(list(range(rows)))
    for idx in (None, index):
        lib.quantize_grouped(x, o, ts, lib.SR, 1, 2, row=lib.Quantized(bufs[0][1], bufs[1][1], ts),
                             col=lib.Quantized(bufs[2][1], bufs[3][1], ts), index=idx, amax=dev_scalar(0.0))
    a, w = rand_operand(rows, K, 5), rand_weights(E, N, K, 6)
    y, z = guarded((rows, N), torch.bfloat16), guarded((rows, N), torch.float32)
    lib.gemm_grouped_fprop(a, w, o, y[1])
    lib.gemm_weight_only(x, w, z[1], offsets=o)
    lib.gemm_weight_only(x[:1], w, z[1][:1], offsets=o)
    dw = guarded((E, 32, N), torch.float32)
    lib.gemm_grouped_wgrad(rand_operand(32, P, 7), rand_operand(N, P, 8), o, dw[1])
    torch.cuda.synchronize()
    for whole, _, pad in (*bufs, y, z, dw):
        assert bool((whole[:pad] == 77).all()) and bool((whole[-pad:] == 77).all())
