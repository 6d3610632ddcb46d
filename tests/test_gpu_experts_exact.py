"""GPU tests of the routed experts' operators on values that come out exactly, and of
their largest counts: gradients against differences without a rounding anywhere, weight
gradients bit for bit, and random words whose call numbers pass 2^32."""

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as lib
from devhelpers import dev_bf16, dev_scalar, fresh_ts, host
from oracle import experts as ox
from oracle import quantize
from test_gpu_experts import dev_i32, dev_operand, empty_result, grouped_buffers, offsets_of
from workloads import random_bf16, to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[20, 0, 35], [16, 129, 1, 0, 3]])
def test_gradients_are_exact_differences(cuda_device, counts):
    """L = sum(dY * Y) is linear in X and in W.  Every block of 16 of every operand holds a 6 and is otherwise on
    E2M1's grid, so under the tensor scale 1 its scale is 1 and nothing is rounded: the differences of L along single
    elements are dX and dW times the step, and all numbers are multiples of 1/8 below 2^18 (exact in fp32)."""
    rng = np.random.default_rng(sum(counts))
    d_in, d_out, E = 32, 48, len(counts)
    off = offsets_of(counts)
    T = int(off[-1])
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=np.float32)
    sixes = lambda shape: np.where(rng.random(shape) < 0.5, 6.0, -6.0).astype(np.float32)  # noqa: E731

    def by_expert(cols):  # a 6 in every block of a row, and in every 16 rows from each expert's first row on
        v = grid[rng.integers(0, len(grid), (T, cols))]
        for b, n, _, _ in ox.spans(off):
            v[b:b + n:16] = sixes(v[b:b + n:16].shape)
        v[:, ::16] = sixes(v[:, ::16].shape)
        return v

    def weights():
        v = grid[rng.integers(0, len(grid), (E, d_out, d_in))]
        v[:, ::16], v[:, :, ::16] = sixes(v[:, ::16].shape), sixes(v[:, :, ::16].shape)
        return v

    one, o = dev_scalar(1.0), dev_i32(off)
    X, G, W = by_expert(d_in), by_expert(d_out), weights()

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

    (xr, xc), (gr, gc), (wr, wc) = operand_pair(X), operand_pair(G), weight_pair(W)
    y, dx, dw = empty_result((T, d_out), False), empty_result((T, d_in), False), empty_result((E, d_out, d_in), False)
    lib.gemm_grouped_fprop(xr, wr, o, y)
    lib.gemm_grouped_dgrad(gr, wc, o, dx)
    lib.gemm_grouped_wgrad(gc, xc, o, dw)
    y, dx, dw = host(y), host(dx), host(dw)
    for g, (b, n, _, _) in enumerate(ox.spans(off)):  # the formulas, on the values before quantization
        x, d, w = X[b:b + n].astype(np.float64), G[b:b + n].astype(np.float64), W[g].astype(np.float64)
        assert np.array_equal(y[b:b + n], x @ w.T) and np.array_equal(dx[b:b + n], d @ w)
        assert np.array_equal(dw[g], d.T @ x)
    base = loss(X, W)
    free = lambda i, b: (i - b) % 16 != 0  # noqa: E731
    for g, (b, n, _, _) in enumerate(ox.spans(off)):
        for i in {b + 1, b + n // 2, b + n - 1} & set(range(b, b + n)):  # rows whose blocks keep their 6
            j = int(rng.integers(1, 16))
            if free(i, b):
                V = X.copy()
                V[i, j] = 0.0 if X[i, j] else 1.0
                assert loss(V, W) - base == float(dx[i, j]) * float(V[i, j] - X[i, j])
        i, j = int(rng.integers(1, 16)) + 16 * (g % 3), int(rng.integers(1, 16)) + 16 * (g % 2)
        V = W.copy()
        V[g, i, j] = 0.0 if W[g, i, j] else 1.0
        assert loss(X, V) - base == float(dw[g, i, j]) * float(V[g, i, j] - W[g, i, j])


@pytest.mark.parametrize("counts,M,N", [([300, 0, 31, 64, 100], 80, 272), ([1000, 1, 40], 130, 70), ([500, 700], 1700, 1300)])
def test_wgrad_exact_sums(cuda_device, counts, M, N):
    """Codes times scales of 1 to 4: partial sums are multiples of 1/4 below 2^20, so any order gives the same bits."""
    rng = np.random.default_rng(9)
    off = offsets_of(counts)
    rows = int(off[-1])
    g = [to_bf16_bits(rng.integers(-4, 5, (rows, n)).astype(np.float32)) for n in (M, N)]
    q = [(*ox.quantize_col(b, off, np.float32(1.0 / 6.0))[:2], np.float32(1.0)) for b in g]
    want, _ = ox.gemm_wgrad(q[0], 1.0, q[1], 1.0, off)
    for bf16 in (False, True):
        dw = empty_result((len(counts), M, N), bf16)
        lib.gemm_grouped_wgrad(dev_operand(q[0]), dev_operand(q[1]), dev_i32(off), dw)
        got = host(dw.float())
        if bf16:
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want)).all()
        else:
            assert np.array_equal(got, want.astype(np.float32))


def test_most_experts_and_random_words_past_2_32(cuda_device):
    """65536 experts of which the first and last have rows: a transposed operand of more than 2^35 elements, whose last
    columns draw words of call numbers past 2^32."""
    import torch

    E, cols = 65536, 4112
    counts = np.zeros(E, dtype=np.int64)
    counts[[0, 1, E - 2, E - 1]] = 40, 3, 130, 127
    off = offsets_of(counts)
    rows = int(off[-1])
    P = lib.rows_padded(rows, E)
    assert cols * P >= 1 << 35
    bits = random_bf16((rows, cols), 6, "gradient")
    ts = fresh_ts(bits)
    tsd, u8 = dev_scalar(ts), dict(dtype=torch.uint8, device="cuda")
    row = lib.empty_quantized(rows, cols, tsd)
    col = lib.Quantized(torch.zeros((cols, P // 2), **u8), torch.zeros((cols, P // 16), **u8), tsd)
    lib.quantize_grouped(dev_bf16(bits), dev_i32(off), tsd, lib.SR, 2 ** 63 + 5, 7, row=row, col=col)
    codes, scales = quantize.quantize_blockscale(bits, ts, 1, 2 ** 63 + 5, 7, 0)
    assert np.array_equal(host(row.codes), codes) and np.array_equal(host(row.scales), scales)
    spans = {g: s for g, s in enumerate(ox.spans(off)) if s[1]}
    assert max((4111 * P + p) >> 3 for _, _, p, _ in spans.values()) >= 1 << 32
    for c in (0, 4100, cols - 1):  # one column of x is one row of the operand
        wide = np.zeros((1, P), dtype=np.float32)
        for b, n, p, _ in spans.values():
            wide[0, p:p + n] = (bits[b:b + n, c].astype(np.uint32) << 16).view(np.float32)
        codes, scales = quantize._quantize_rows(wide, np.float32(ts), 1, 2 ** 63 + 5, 7, 1, P, np.array([c]))
        got_codes, got_scales = host(col.codes[c]), host(col.scales[c])
        for b, n, p, width in spans.values():
            assert np.array_equal(got_codes[p // 2:(p + width) // 2], codes[0, p // 2:(p + width) // 2])
            assert np.array_equal(got_scales[p // 16:(p + width) // 16], scales[0, p // 16:(p + width) // 16])
    # the products of the last expert alone, by its own tensor scale
    N, K = 24, 32
    w = lib.ExpertWeights(torch.full((E, N, K // 2), 0x22, **u8), torch.full((E, N, K // 16), 0x78, **u8),
                          torch.arange(1, E + 1, dtype=torch.float32, device="cuda"))
    a = lib.Quantized(torch.full((rows, K // 2), 0x22, **u8), torch.full((rows, K // 16), 0x78, **u8), dev_scalar(1.0))
    x = torch.ones((rows, K), dtype=torch.bfloat16, device="cuda")
    owner = torch.from_numpy(np.repeat(np.arange(1, E + 1), counts).astype(np.float32)).cuda()
    for call in (lambda y: lib.gemm_grouped_fprop(a, w, dev_i32(off), y), lambda y: lib.gemm_weight_only(x, w, y, offsets=dev_i32(off))):
        y = empty_result((rows, N), False)
        call(y)
        assert torch.equal(y, (32.0 * owner)[:, None].expand(rows, N))


def test_row_wise_random_words_past_2_32(cuda_device):
    """More than 2^35 elements row by row, gathered from a few tokens."""
    import torch

    cols, tokens = 4112, 64
    rows = (1 << 35) // cols + 300
    bits = random_bf16((tokens, cols), 8, "gradient")
    ts = fresh_ts(bits)
    index = torch.randint(0, tokens, (rows,), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    q = lib.empty_quantized(rows, cols, dev_scalar(ts))
    lib.quantize_grouped(dev_bf16(bits), dev_i32([0, 5, rows]), q.ts, lib.SR, 77, 2 ** 31 + 3, row=q, index=index)
    ids = np.array([0, 4, 5, 31, 32, rows // 2, rows - 290, rows - 33, rows - 1])
    assert (int(ids[-2]) * cols) >> 3 >= 1 << 32
    x = (bits[index[torch.from_numpy(ids).cuda()].cpu().numpy()].astype(np.uint32) << 16).view(np.float32)
    codes, scales = quantize._quantize_rows(x, np.float32(ts), 1, 77, 2 ** 31 + 3, 0, cols, ids)
    at = torch.from_numpy(ids).cuda()
    assert np.array_equal(host(q.codes[at]), codes) and np.array_equal(host(q.scales[at]), scales)
