"""GPU tests of the routed experts' operators against the numpy oracle.

Quantizer: codes, scale bytes and amax bit for bit.  Products: within 1e-5 * |ts|
* sum |a b| of the fp64 definition (the library's bar), bf16 results half a step
(2^-8 of the value) further, and bit for bit on operands whose partial sums fp32
holds exactly.  What belongs to no expert has to stay as it was.
"""

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as lib
from devhelpers import dev_bf16, dev_scalar, fresh_ts, host
from oracle import experts as ox
from oracle import formats, quantize
from workloads import random_bf16, to_bf16_bits

pytestmark = pytest.mark.gpu

SENTINEL = 0xA5


def dev_i32(values):
    import torch

    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def offsets_of(counts, before=0):
    return np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int64)


def filled(shape):
    import torch

    return torch.full(shape, SENTINEL, dtype=torch.uint8, device="cuda")


def grouped_buffers(rows, cols, experts, ts, row=True, col=True):
    P = lib.rows_padded(rows, experts)
    r = lib.Quantized(filled((rows, cols // 2)), filled((rows, cols // 16)), ts) if row else None
    c = lib.Quantized(filled((cols, P // 2)), filled((cols, P // 16)), ts) if col else None
    return r, c


def check_row(q, bits, offsets, ts, rounding, seed, offset):
    codes, scales, owned = ox.quantize_row(bits, offsets, ts, rounding, seed, offset)
    gc, gs = host(q.codes), host(q.scales)
    assert np.array_equal(gs[owned], scales[owned]) and np.array_equal(gc[owned], codes[owned])
    assert (gc[~owned] == SENTINEL).all() and (gs[~owned] == SENTINEL).all()


def check_col(q, bits, offsets, ts, rounding, seed, offset):
    codes, scales, written = ox.quantize_col(bits, offsets, ts, rounding, seed, offset)
    gc, gs = host(q.codes), host(q.scales)
    wide = np.repeat(written, 8)
    assert np.array_equal(gs[:, written], scales[:, written]) and np.array_equal(gc[:, wide], codes[:, wide])
    assert (gc[:, ~wide] == SENTINEL).all() and (gs[:, ~written] == SENTINEL).all()


# ----------------------------------------------------------------- quantizer --

COUNTS = [
    ([1], 0, 0),
    ([128], 0, 0),
    ([0, 5, 0, 0, 129, 64, 1, 0], 0, 0),
    ([127, 128, 129, 255, 16, 17], 3, 9),     # rows before the first expert and behind the last
    ([0, 0, 0], 0, 7),                        # rows, but no expert's
    ([3] * 70, 0, 0),                         # more experts than lanes of a wave
    ([0] * 64 + [40] + [0] * 64 + [2], 1, 1),
]


@pytest.mark.parametrize("rounding", [lib.RNE, lib.SR])
@pytest.mark.parametrize("cols", [16, 272, 528])
@pytest.mark.parametrize("counts,before,behind", COUNTS)
def test_quantize_grouped(cuda_device, counts, before, behind, cols, rounding):
    off = offsets_of(counts, before)
    rows = int(off[-1]) + behind
    bits = random_bf16((rows, cols), 5 + cols, "gradient")
    ts = fresh_ts(bits)
    tsd, amax = dev_scalar(ts), dev_scalar(0.0)
    for row, col in ((True, True), (True, False), (False, True)):
        qr, qc = grouped_buffers(rows, cols, len(counts), tsd, row, col)
        lib.quantize_grouped(dev_bf16(bits), dev_i32(off), tsd, rounding, 2 ** 63 + 5, 2 ** 31 + 1, row=qr, col=qc,
                             amax=amax)
        if row:
            check_row(qr, bits, off, ts, rounding, 2 ** 63 + 5, 2 ** 31 + 1)
        if col:
            check_col(qc, bits, off, ts, rounding, 2 ** 63 + 5, 2 ** 31 + 1)
        want = ox.amax(bits, off) if sum(counts) else np.float32(0)
        assert host(amax)[0] == want


@pytest.mark.parametrize("rounding", [lib.RNE, lib.SR])
def test_quantize_grouped_index_and_strides(cuda_device, rounding):
    """Rows gathered from a wider tensor: repeated, in any order, and out of range (zeros)."""
    x = random_bf16((37, 160 + 32), 3, "heavy")
    counts = [40, 0, 21, 130]
    off = offsets_of(counts)
    rng = np.random.default_rng(1)
    index = rng.integers(0, 37, off[-1])
    index[[0, 45, 100]] = [-1, 37, 2 ** 31 - 1]
    index[-1] = -2 ** 31
    wide = dev_bf16(x)
    view = wide[:, 16:176]  # row stride 192, base 32 bytes in
    bits = ox.gather(np.ascontiguousarray(x[:, 16:176]), index)
    ts = fresh_ts(bits)
    tsd, amax = dev_scalar(ts), dev_scalar(0.0)
    qr, qc = grouped_buffers(len(index), 160, 4, tsd)
    lib.quantize_grouped(view, dev_i32(off), tsd, rounding, 7, 3, row=qr, col=qc, index=dev_i32(index), amax=amax)
    check_row(qr, bits, off, ts, rounding, 7, 3)
    check_col(qc, bits, off, ts, rounding, 7, 3)
    assert host(amax)[0] == ox.amax(bits, off)


def test_quantize_grouped_amax_only_and_running(cuda_device):
    bits = random_bf16((50, 64), 2)
    off = offsets_of([10, 0, 30], 4)
    amax = dev_scalar(0.0)
    lib.quantize_grouped(dev_bf16(bits), dev_i32(off), None, amax=amax)
    assert host(amax)[0] == ox.amax(bits, off)
    amax = dev_scalar(1000.0)
    lib.quantize_grouped(dev_bf16(bits), dev_i32(off), None, amax=amax)
    assert host(amax)[0] == 1000.0
    big = bits.copy()
    big[0] = big[-1] = 0x7FC0  # NaN in rows of no expert
    amax = dev_scalar(0.0)
    lib.quantize_grouped(dev_bf16(big), dev_i32(off), None, amax=amax)
    assert host(amax)[0] == ox.amax(bits, off)
    big[20, 3] = 0x7FC0
    lib.quantize_grouped(dev_bf16(big), dev_i32(off), None, amax=amax)
    assert np.isnan(host(amax)[0])


@pytest.mark.parametrize("ts", [1e-3, 1e-38, 1e30, 3e38, 0.0])
@pytest.mark.parametrize("rounding", [lib.RNE, lib.SR])
def test_quantize_grouped_special_values(cuda_device, ts, rounding):
    """NaN, infinities, zeros of both signs, subnormals and blocks of one magnitude, under ordinary and extreme scales."""
    bits = random_bf16((96, 64), 11, "logrange")
    bits[0, 5], bits[3, 20], bits[40, 63], bits[41, 0] = 0x7FC1, 0x7F80, 0xFF80, 0xFFC0
    bits[10, :16], bits[11, :16], bits[12, 16:32] = 0, 0x8000, 0x0001
    off = offsets_of([33, 0, 63])
    tsd = dev_scalar(ts)
    qr, qc = grouped_buffers(96, 64, 3, tsd)
    lib.quantize_grouped(dev_bf16(bits), dev_i32(off), tsd, rounding, 1, 2, row=qr, col=qc)
    with np.errstate(all="ignore"):
        check_row(qr, bits, off, np.float32(ts), rounding, 1, 2)
        check_col(qc, bits, off, np.float32(ts), rounding, 1, 2)


# ------------------------------------------------------------------ products --

def operand(shape, seed, kind="normal"):
    """(codes, scales) by the oracle, its tensor scale, and the device operand."""
    bits = random_bf16(shape, seed, kind)
    ts = fresh_ts(bits)
    codes, scales = quantize.quantize_blockscale(bits, ts)
    return codes, scales, ts


def dev_u8(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_operand(q):
    return lib.Quantized(dev_u8(q[0]), dev_u8(q[1]), dev_scalar(q[2]))


def weights(experts, N, K, seed, one_ts=False):
    import torch

    parts = [operand((N, K), seed + g) for g in range(experts)]
    ts = np.array([parts[0 if one_ts else g][2] for g in range(experts)], dtype=np.float32)
    codes, scales = np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])
    return codes, scales, ts, lib.ExpertWeights(dev_u8(codes), dev_u8(scales),
                                                torch.from_numpy(ts[:1].copy() if one_ts else ts).cuda())


def empty_result(shape, bf16):
    import torch

    return torch.full(shape, -77.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")


def check_result(out, ref, bound, owned=None, bf16=False):
    got = out.float().cpu().numpy().astype(np.float64)
    if owned is not None:
        assert (got[~owned] == -77.0).all(), "rows of no expert changed"
        got, ref, bound = got[owned], ref[owned], bound[owned]
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan)
    lim = 1e-5 * bound
    if bf16:  # half a step of the value before rounding, which is within lim of ref
        lim = lim + 2.0 ** -8 * (np.abs(ref) + lim)
    err = np.abs(got - ref)
    assert (err[~nan] <= lim[~nan]).all(), (err[~nan] - lim[~nan]).max()


# every height of tile: 1 .. 32, 33 .. 64, 65 .. 128, 129 .. 256 rows, and rests behind full tiles
TILES = [([1], 0, 0), ([32, 33, 0, 64, 65], 0, 0), ([128, 129], 2, 3), ([255, 256, 257], 0, 1), ([300, 0, 7, 600], 0, 0),
         ([2] * 67, 1, 2), ([0, 0], 0, 5)]


@pytest.mark.parametrize("K", [16, 128, 400])
@pytest.mark.parametrize("N", [1, 37, 300])
@pytest.mark.parametrize("counts,before,behind", TILES)
def test_gemm_grouped_rows(cuda_device, counts, before, behind, N, K):
    off = offsets_of(counts, before)
    rows, E = int(off[-1]) + behind, len(counts)
    a = operand((rows, K), 40 + K, "heavy" if K > 16 else "normal")
    bc, bs, bts, w = weights(E, N, K, 50, one_ts=N == 37)
    ref, bound, owned = ox.gemm_rows(a, a[2], bc, bs, bts, off)
    y = empty_result((rows, N), False)
    lib.gemm_grouped_fprop(dev_operand(a), w, dev_i32(off), y)
    check_result(y, ref, bound, owned)
    y16, amax = empty_result((rows, N), True), dev_scalar(0.0)
    lib.gemm_grouped_dgrad(dev_operand(a), w, dev_i32(off), y16, amax=amax)
    check_result(y16, ref, bound, owned, bf16=True)
    stored = y16.float().cpu().numpy()[owned]
    assert host(amax)[0] == (np.abs(stored).max() if stored.size else 0.0)


def test_gemm_grouped_empty_contraction_and_sizes(cuda_device):
    import torch

    off = dev_i32([0, 3, 5])
    a = lib.Quantized(torch.empty((6, 0), dtype=torch.uint8, device="cuda"),
                      torch.empty((6, 0), dtype=torch.uint8, device="cuda"), dev_scalar(1.0))
    w = lib.empty_expert_weights(2, 9, 0, dev_scalar(1.0))
    y = empty_result((6, 9), False)
    lib.gemm_grouped_fprop(a, w, off, y)
    got = y.cpu().numpy()
    assert (got[:5] == 0).all() and (got[5] == -77.0).all()
    lib.gemm_grouped_fprop(lib.Quantized(a.codes[:0], a.scales[:0], a.ts), w, dev_i32([0, 0, 0]), y[:0])
    lib.gemm_weight_only(torch.empty((3, 0), dtype=torch.bfloat16, device="cuda"), w.expert(0), y[:3])
    assert (y.cpu().numpy()[:3] == 0).all()


@pytest.mark.parametrize("counts,before,behind", [([1], 0, 0), ([16, 0, 129], 0, 0), ([128, 300, 0, 5], 3, 2), ([4] * 66, 0, 0)])
@pytest.mark.parametrize("M,N", [(16, 16), (48, 300), (272, 37), (300, 260)])
@pytest.mark.parametrize("bf16", [False, True])
def test_gemm_grouped_wgrad(cuda_device, counts, before, behind, M, N, bf16):
    import torch

    off = offsets_of(counts, before)
    rows, E = int(off[-1]) + behind, len(counts)
    P = ox.rows_padded(rows, E)
    ops, dev = [], []
    for width, seed in ((M, 60), (N, 61)):
        bits = random_bf16((rows, width), seed)
        ts = fresh_ts(bits)
        codes, scales, written = ox.quantize_col(bits, off, ts)
        ops.append((codes, scales, ts))
        codes, scales = codes.copy(), scales.copy()
        codes[:, ~np.repeat(written, 8)], scales[:, ~written] = 0x77, 0xFF  # what no expert owns is not read
        dev.append(lib.Quantized(dev_u8(codes), dev_u8(scales), dev_scalar(ts)))
        assert codes.shape == (width, P // 2)
    ref, bound = ox.gemm_wgrad(ops[0], ops[0][2], ops[1], ops[1][2], off)
    dw = empty_result((E, M, N), bf16)
    lib.gemm_grouped_wgrad(dev[0], dev[1], dev_i32(off), dw)
    check_result(dw, ref, bound, bf16=bf16)
    assert (dw[torch.tensor([n == 0 for n in counts])] == 0).all()


def exact_operand(rng, rows, cols):
    """Small integers as codes with scale 1 (UE5M3 0x78): every partial sum is an integer below 2^24."""
    codes = rng.integers(0, 16, (rows, cols // 2)).astype(np.uint8) | (rng.integers(0, 16, (rows, cols // 2)) << 4).astype(np.uint8)
    return codes, np.full((rows, cols // 16), 0x78, dtype=np.uint8), np.float32(1.0)


def test_products_exact_sums(cuda_device):
    """Products whose partial sums are multiples of 1/4 below 2^22: any order of summation gives the same bits."""
    import torch

    rng = np.random.default_rng(9)
    counts, N, K = [300, 0, 31, 64, 100], 270, 2064
    off = offsets_of(counts)
    a = exact_operand(rng, int(off[-1]), K)
    parts = [exact_operand(rng, N, K) for _ in counts]
    bc, bs = np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts])
    w = lib.ExpertWeights(dev_u8(bc), dev_u8(bs), dev_scalar(1.0))
    ref, _, _ = ox.gemm_rows(a, 1.0, bc, bs, [1.0] * 5, off)
    y = empty_result(ref.shape, False)
    lib.gemm_grouped_fprop(dev_operand(a), w, dev_i32(off), y)
    assert np.array_equal(host(y), ref.astype(np.float32))
    # the same values as bf16 tokens
    x = to_bf16_bits(quantize.dequantize_unscaled(a[0], a[1]))
    y = empty_result(ref.shape, False)
    lib.gemm_weight_only(dev_bf16(x), w, y, offsets=dev_i32(off))
    assert np.array_equal(host(y), ref.astype(np.float32))
    # and as transposed operands
    rows = int(off[-1])
    g = [to_bf16_bits(rng.integers(-4, 5, (rows, n)).astype(np.float32)) for n in (80, 272)]
    q = [ox.quantize_col(b, off, np.float32(1.0 / 6.0)) for b in g]  # any scale: values are what the codes say
    ts = np.float32(1.0)
    refw, _ = ox.gemm_wgrad(q[0], ts, q[1], ts, off)
    dw = empty_result((5, 80, 272), False)
    lib.gemm_grouped_wgrad(lib.Quantized(dev_u8(q[0][0]), dev_u8(q[0][1]), dev_scalar(ts)),
                           lib.Quantized(dev_u8(q[1][0]), dev_u8(q[1][1]), dev_scalar(ts)), dev_i32(off), dw)
    assert np.allclose(host(dw), refw, rtol=1e-6, atol=0)
    torch.cuda.synchronize()


def test_every_scale_and_code_through_the_products(cuda_device):
    """Each (code, scale byte) pair against a unit token: the exact value, NaN for 0xFF."""
    codes = np.zeros((256, 16), dtype=np.uint8)      # row = scale byte, column = one code per block of 16
    N, K = 256, 256
    codes = np.zeros((N, K // 2), dtype=np.uint8)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], K // 16, 1)
    for b in range(16):                              # block b holds code b at place b
        codes[:, 8 * b + b // 2] = b << (4 * (b & 1))
    x = np.zeros((16, K), dtype=np.float32)
    for b in range(16):
        x[b, 16 * b + b] = 1.0
    want = np.zeros((16, N))
    for b in range(16):
        want[b] = formats.e2m1_decode(np.full(N, b, dtype=np.uint8)) * formats.ue5m3_decode(np.arange(256, dtype=np.uint8))
    want[:, 255] = np.nan
    out = empty_result((16, N), False)
    w = lib.Quantized(dev_u8(codes), dev_u8(scales), dev_scalar(1.0))
    lib.gemm_weight_only(dev_bf16(to_bf16_bits(x)), w, out)
    assert np.array_equal(host(out), want.astype(np.float32), equal_nan=True)
    one = empty_result((1, N), False)
    for b in range(16):
        lib.gemm_weight_only(dev_bf16(to_bf16_bits(x[b:b + 1])), w, one)
        assert np.array_equal(host(one)[0], want[b].astype(np.float32), equal_nan=True)
    # the same through the quantized product
    xc, xs = quantize.quantize_blockscale(to_bf16_bits(x * 6), np.float32(1.0))
    y = empty_result((16, N), False)
    lib.gemm_grouped_fprop(lib.Quantized(dev_u8(xc), dev_u8(xs), dev_scalar(1.0 / 6)),
                           lib.ExpertWeights(w.codes[None], w.scales[None], w.ts), dev_i32([0, 16]), y)
    got, ref = host(y).astype(np.float64), want
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref)[ok] <= 2.0 ** -22 * np.abs(ref)[ok]).all()  # ts 1/6 rounded, and two multiplications


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 16, 17, 33, 64, 70])
@pytest.mark.parametrize("N,K", [(1, 16), (37, 400), (64, 256), (300, 2064), (1305, 512)])
def test_weight_only_dense(cuda_device, rows, N, K):
    bits = random_bf16((rows, K), 3, "heavy" if K > 16 else "normal")
    q = operand((N, K), 4)
    ref, bound, _ = ox.weight_only(bits, q[0][None], q[1][None], [q[2]], [0, rows])
    for bf16 in (False, True):
        out = empty_result((rows, N), bf16)
        lib.gemm_weight_only(dev_bf16(bits), dev_operand(q), out)
        check_result(out, ref, bound, bf16=bf16)


@pytest.mark.parametrize("counts,before,behind", [([1], 0, 0), ([1, 0, 1, 1, 0, 2], 0, 0), ([16, 17, 0, 64, 65, 3], 1, 2),
                                                  ([1] * 70, 0, 0), ([0] * 100 + [9, 2], 0, 1), ([0, 0], 0, 3)])
@pytest.mark.parametrize("N,K", [(37, 400), (300, 512)])
def test_weight_only_experts(cuda_device, counts, before, behind, N, K):
    off = offsets_of(counts, before)
    rows = int(off[-1]) + behind
    bits = random_bf16((rows, K), 3)
    bc, bs, bts, w = weights(len(counts), N, K, 70, one_ts=N == 37)
    ref, bound, owned = ox.weight_only(bits, bc, bs, bts, off)
    for bf16 in (False, True):
        out = empty_result((rows, N), bf16)
        lib.gemm_weight_only(dev_bf16(bits), w, out, offsets=dev_i32(off))
        check_result(out, ref, bound, owned, bf16=bf16)


def test_weight_only_strides_and_special_values(cuda_device):
    import torch

    K, N, rows = 272, 45, 6
    bits = random_bf16((rows, K + 40), 8)
    bits[1, 20], bits[2, 30], bits[3, 40] = 0x7FC0, 0x7F80, 0xFF80  # in the view: NaN, Inf, -Inf tokens
    q = operand((N, K), 9)
    codes, scales = q[0].copy(), q[1].copy()
    scales[7, 3] = 0xFF                     # a NaN block in weight row 7
    codes[:, (30 - 8) // 2], codes[:, (40 - 8) // 2] = 0x55, 0x55  # the infinities meet positive weights
    scales[:, (30 - 8) // 16] = np.where(scales[:, (30 - 8) // 16] == 0, 0x40, scales[:, (30 - 8) // 16])
    scales[:, (40 - 8) // 16] = np.where(scales[:, (40 - 8) // 16] == 0, 0x40, scales[:, (40 - 8) // 16])
    view = dev_bf16(bits)[:, 8:8 + K]
    ref, bound, _ = ox.weight_only(np.ascontiguousarray(bits[:, 8:8 + K]), codes[None], scales[None], [q[2]], [0, rows])
    wide = torch.full((rows, N + 11), -77.0, device="cuda")
    lib.gemm_weight_only(view, lib.Quantized(dev_u8(codes), dev_u8(scales), dev_scalar(q[2])), wide[:, :N])
    got = wide.cpu().numpy()
    assert (got[:, N:] == -77.0).all()
    got = got[:, :N].astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.isnan(got[:, 7]).all() and np.isnan(got[1]).all()
    inf = np.isinf(ref)
    assert inf[2, :7].all() and np.array_equal(got[inf], ref[inf])
    ok = np.isfinite(ref)
    assert (np.abs(got[ok] - ref[ok]) <= 1e-5 * bound[ok]).all()


# ------------------------------------------------------------- used together --

def test_training_step_of_routed_experts(cuda_device):
    """Quantize (gathered tokens, weights, stochastic gradient), fprop, dgrad, wgrad and the scale refresh, as a step
    makes them, against the oracle's own quantization of the same inputs."""
    import torch

    tokens, d_in, d_out, E = 70, 144, 96, 5
    rng = np.random.default_rng(4)
    routed = [np.sort(rng.choice(tokens, n, replace=False)) for n in (50, 0, 33, 1, 56)]
    off, index = offsets_of([len(r) for r in routed]), np.concatenate(routed)
    T = len(index)
    X, G = random_bf16((tokens, d_in), 1), random_bf16((T, d_out), 2, "gradient")
    Wb = random_bf16((E * d_out, d_in), 3).reshape(E, d_out, d_in)
    o, idx = dev_i32(off), dev_i32(index)
    x, dy, wd = dev_bf16(X), dev_bf16(G), dev_bf16(Wb.reshape(E * d_out, d_in)).view(E, d_out, d_in)

    def refreshed(run):
        amax, ts = dev_scalar(0.0), dev_scalar(1.0)
        run(amax)
        lib.update_tensor_scale(amax, ts, 0, 1)
        return ts

    ts_x = refreshed(lambda m: lib.quantize_grouped(x, o, None, index=idx, amax=m))
    ts_g = refreshed(lambda m: lib.quantize_grouped(dy, o, None, amax=m))
    ts_w = torch.cat([refreshed(lambda m, e=e: lib.quantize_blockscale(wd[e], None, amax=m)) for e in range(E)])
    wr, wc = lib.empty_expert_weights(E, d_out, d_in, ts_w), lib.empty_expert_weights(E, d_in, d_out, ts_w)
    for e in range(E):
        lib.quantize_blockscale(wd[e], ts_w[e:e + 1], row=wr.expert(e), col=wc.expert(e))
    xr, xc = grouped_buffers(T, d_in, E, ts_x)
    gr, gc = grouped_buffers(T, d_out, E, ts_g)
    amax = dev_scalar(0.0)
    lib.quantize_grouped(x, o, ts_x, row=xr, col=xc, index=idx, amax=amax)
    lib.quantize_grouped(dy, o, ts_g, lib.SR, 99, 5, row=gr, col=gc)
    y, dx, dw = empty_result((T, d_out), False), empty_result((T, d_in), False), empty_result((E, d_out, d_in), False)
    lib.gemm_grouped_fprop(xr, wr, o, y)
    lib.gemm_grouped_dgrad(gr, wc, o, dx)
    lib.gemm_grouped_wgrad(gc, xc, o, dw)

    Xg = ox.gather(X, index)
    tx, tg = fresh_ts(Xg), fresh_ts(G)
    tw = [fresh_ts(Wb[e]) for e in range(E)]
    assert host(ts_x)[0] == tx and host(ts_g)[0] == tg and np.array_equal(host(ts_w), np.array(tw))
    check_row(xr, Xg, off, tx, 0, 0, 0)
    check_col(gc, G, off, tg, 1, 99, 5)
    owr = [quantize.quantize_blockscale(Wb[e], tw[e]) for e in range(E)]
    owc = [quantize.quantize_blockscale(Wb[e], tw[e], orientation=1) for e in range(E)]
    oxr, oxc = ox.quantize_row(Xg, off, tx), ox.quantize_col(Xg, off, tx)
    ogr, ogc = ox.quantize_row(G, off, tg, 1, 99, 5), ox.quantize_col(G, off, tg, 1, 99, 5)
    stack = lambda q: (np.stack([c for c, _ in q]), np.stack([s for _, s in q]))  # noqa: E731
    check_result(y, *ox.gemm_rows(oxr, tx, *stack(owr), tw, off))
    check_result(dx, *ox.gemm_rows(ogr, tg, *stack(owc), tw, off))
    check_result(dw, *ox.gemm_wgrad(ogc, tg, oxc, tx, off))
    # a generation step with the same weights: the tokens in bf16
    out = empty_result((T, d_out), False)
    lib.gemm_weight_only(x[idx.long()].contiguous(), wr, out, offsets=o)
    check_result(out, *ox.weight_only(Xg, *stack(owr), tw, off))


def test_gradients_against_differences(cuda_device):
    """With L = sum(dY * Y) the forward pass is linear in X and W: on operands that FP4 holds exactly, the differences of
    L along single elements are dX and dW exactly (sums of small multiples of 1/2)."""
    rng = np.random.default_rng(12)
    counts, d_in, d_out = [20, 0, 35], 32, 48
    off, E, T = offsets_of(counts), 3, 55
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=np.float32)

    def exact(shape):  # every row and column block of 16 has its largest magnitude 6: scale 1 under ts = 1
        v = grid[rng.integers(0, len(grid), shape)]
        v[..., ::16, :] = np.where(rng.random(v[..., ::16, :].shape) < 0.5, 6, -6)
        v[..., :, ::16] = 6
        return v

    one, o = dev_scalar(1.0), dev_i32(off)
    X, W, G = exact((T, d_in)), exact((E, d_out, d_in)), exact((T, d_out))

    def operand_pair(v):
        q = grouped_buffers(*v.shape, E, one)
        lib.quantize_grouped(dev_bf16(to_bf16_bits(v)), o, one, row=q[0], col=q[1])
        return q

    def weight_pair(v):
        r, c = lib.empty_expert_weights(E, d_out, d_in, one), lib.empty_expert_weights(E, d_in, d_out, one)
        for e in range(E):
            lib.quantize_blockscale(dev_bf16(to_bf16_bits(v[e])), one, row=r.expert(e), col=c.expert(e))
        return r, c

    def loss(x, w):
        y = empty_result((T, d_out), False)
        lib.gemm_grouped_fprop(operand_pair(x)[0], weight_pair(w)[0], o, y)
        return float((host(y).astype(np.float64) * G).sum())

    # the transposed blocks hold a 6 only where a column block starts inside one expert: scales below 1 keep the
    # values of this grid exact as long as the block's amax is a power of two times 6 or its elements fit it
    xr, xc = operand_pair(X)
    gr, gc = operand_pair(G)
    _, wc = weight_pair(W)
    dx, dw = empty_result((T, d_in), False), empty_result((E, d_out, d_in), False)
    lib.gemm_grouped_dgrad(gr, wc, o, dx)
    lib.gemm_grouped_wgrad(gc, xc, o, dw)
    base = loss(X, W)
    for i, j in ((0, 1), (19, 17), (20, 31), (54, 5)):
        Y = X.copy()
        Y[i, j] = 0.0 if X[i, j] else 1.0
        assert loss(Y, W) - base == pytest.approx(float(host(dx)[i, j]) * float(Y[i, j] - X[i, j]), rel=1e-5, abs=1e-3)
    vals = ox.gemm_wgrad((host(gc.codes), host(gc.scales)), 1.0, (host(xc.codes), host(xc.scales)), 1.0, off)[0]
    exact_cols = np.array([[np.array_equal(vals[e], G[b:b + n].T.astype(np.float64) @ X[b:b + n])]
                           for e, (b, n, _, _) in enumerate(ox.spans(off))])
    for e, i, j in ((0, 3, 1), (0, 47, 30), (2, 9, 17)):
        V = W.copy()
        V[e, i, j] = 0.0 if W[e, i, j] else 1.0
        want = (loss(X, V) - base) / float(V[e, i, j] - W[e, i, j])
        if exact_cols[e]:
            assert float(host(dw)[e, i, j]) == pytest.approx(want, rel=1e-5, abs=1e-3)
        else:  # a column block without a 6 is rounded: E2M1's step is at most 1/4 of the value, twice
            b, n = ox.spans(off)[e][:2]
            assert abs(float(host(dw)[e, i, j]) - want) <= 0.5 * (np.abs(G[b:b + n, i]) * np.abs(X[b:b + n, j])).sum()
    assert (host(dw)[1] == 0).all()


def test_readme_examples(cuda_device):
    """The README's blocks run in their order; the experts' results are those of their operands' values."""
    import os

    import torch

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    ns = {}
    for block in text.split("```python\n")[1:]:
        exec(compile(block.split("```")[0], "README.md", "exec"), ns)
    torch.cuda.synchronize()

    def value(q):
        return lib.dequantize(q, torch.empty((q.rows, q.cols), dtype=torch.float32, device="cuda")).double()

    def check(out, a, b, bf16):
        ref, bound = a @ b.t(), 1e-5 * (a.abs() @ b.abs().t())
        assert bool(((out.double() - ref).abs() <= (bound + 2.0 ** -8 * (ref.abs() + bound) if bf16 else bound)).all())

    off = ns["offsets"].tolist()
    x, xt, g, gt = value(ns["Xe"][0]), value(ns["Xe"][1]), value(ns["Ge"][0]), value(ns["Ge"][1])
    for e in range(ns["experts"]):
        b, n = off[e], off[e + 1] - off[e]
        p, w = 128 * (-(-b // 128) + e), value(ns["We"].expert(e))
        check(ns["ye"][b:b + n], x[b:b + n], w, True)
        check(ns["dxe"][b:b + n], g[b:b + n], value(ns["WeT"].expert(e)), False)
        check(ns["dwe"][e], gt[:, p:p + -(-n // 128) * 128], xt[:, p:p + -(-n // 128) * 128], False)
    assert float(ns["yamax"]) == float(ns["ye"].float().abs().max())
    check(ns["y1"], ns["x"][:1].double(), value(ns["W"][0]), True)
    check(ns["y64"], ns["some"].double(), value(ns["We"].expert(0)), True)


@pytest.mark.parametrize("experts", [65, 300, 4200])
def test_many_experts(cuda_device, experts):
    """More experts than one or two rounds of 64 ranges tell apart; few have rows."""
    rng = np.random.default_rng(experts)
    counts = np.where(rng.random(experts) < 0.05, rng.integers(1, 40, experts), 0)
    counts[[0, -1]] = 3, 5
    off = offsets_of(counts, 2)
    rows, N, K = int(off[-1]) + 1, 24, 32
    bits = random_bf16((rows, K), 6, "gradient")
    ts, o = fresh_ts(bits), dev_i32(off)
    tsd, amax = dev_scalar(ts), dev_scalar(0.0)
    qr, qc = grouped_buffers(rows, K, experts, tsd)
    lib.quantize_grouped(dev_bf16(bits), o, tsd, lib.SR, 5, 1, row=qr, col=qc, amax=amax)
    check_row(qr, bits, off, ts, 1, 5, 1)
    check_col(qc, bits, off, ts, 1, 5, 1)
    assert host(amax)[0] == ox.amax(bits, off)
    q = operand((N, K), 7)
    bc, bs, bts = np.repeat(q[0][None], experts, 0), np.repeat(q[1][None], experts, 0), np.arange(1, experts + 1, dtype=np.float32)
    import torch

    w = lib.ExpertWeights(dev_u8(bc), dev_u8(bs), torch.from_numpy(bts).cuda())  # told apart by their tensor scales
    a = quantize.quantize_blockscale(bits, ts)
    y = empty_result((rows, N), False)
    lib.gemm_grouped_fprop(dev_operand((*a, ts)), w, o, y)
    check_result(y, *ox.gemm_rows(a, ts, bc, bs, bts, off))
    y = empty_result((rows, N), False)
    lib.gemm_weight_only(dev_bf16(bits), w, y, offsets=o)
    check_result(y, *ox.weight_only(bits, bc, bs, bts, off))
