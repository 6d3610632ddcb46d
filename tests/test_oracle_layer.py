"""CPU pins of the 8-bit and dropout oracles: torch's float8 casts (library
routines), hand-worked scales, the mask's rate and its independence of layout."""

import numpy as np
import pytest
import torch

from oracle import dropout, fp8, philox

F8 = {fp8.E4M3: torch.float8_e4m3fn, fp8.E5M2: torch.float8_e5m2}


@pytest.mark.parametrize("fmt", [fp8.E4M3, fp8.E5M2])
def test_decode_is_the_format(fmt):
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(F8[fmt]).double().numpy()
    assert np.array_equal(fp8.decode(codes, fmt), ref, equal_nan=True)


@pytest.mark.parametrize("fmt", [fp8.E4M3, fp8.E5M2])
def test_encode_every_midpoint_and_random_values(fmt):
    f = fp8.LARGEST[fmt]
    grid = np.unique(fp8.decode(np.arange(256, dtype=np.uint8), fmt))
    grid = grid[np.isfinite(grid)]
    mid = (grid[:-1] + grid[1:]) / 2
    rng = np.random.default_rng(1)
    v = np.concatenate([grid, mid, np.nextafter(mid.astype(np.float32), np.float32(np.inf)),
                        np.nextafter(mid.astype(np.float32), np.float32(-np.inf)),
                        rng.uniform(-f, f, 100000), rng.standard_normal(100000) * 2.0 ** rng.integers(-18, 5, 100000),
                        [0.0, -0.0]]).astype(np.float32)
    ref = torch.from_numpy(v).to(F8[fmt]).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(v, fmt), ref)


def test_block_scales_worked():
    s, r = fp8.block_scale(np.float32([448.0, 7.0, 0.0, 2.0 ** -133, np.inf, np.nan]), fp8.E4M3, False)
    assert s[0] == 1.0 and s[1] == 0.015625 and s[2] == s[3] == np.float32(2.0 ** -126)
    assert r[0] == 1.0 and r[1] == 64.0 and r[2] == np.float32(2.0 ** 126)
    assert np.isnan(s[4:]).all()
    # exact powers of two stay, everything else rounds up; the smallest scale is 2^-127
    a = np.float32([448.0, 449.0, 447.0, 896.0, 0.0, 2.0 ** -133, np.inf])
    s, r = fp8.block_scale(a, fp8.E4M3, True)
    assert s.tolist() == [127, 128, 127, 128, 0, 0, 255]
    assert np.array_equal(r[:6], np.exp2(127.0 - s[:6]).astype(np.float32))


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("e8m0", [False, True])
def test_quantize_layout_and_error(tile, e8m0):
    from workloads import random_bf16

    bits = random_bf16((200, 300), 5, "heavy")
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).double().numpy()
    for o, xo in ((0, x), (1, x.T)):
        codes, scales = fp8.quantize(bits, fp8.E4M3, e8m0, tile, o)
        R, C = xo.shape
        nb = -(-C // 128)
        assert codes.shape == (R, nb * 128) and scales.shape == (nb, -(-R // 128) if tile else R)
        assert not codes[:, C:].any()
        v = fp8.operand(codes, scales, fp8.E4M3, tile)[:, :C]
        s = fp8.scale_values(scales)
        s = (s[:, np.arange(R) // 128] if tile else s).T.repeat(128, 1)[:, :C]
        # half a step of the value's binade (2^-4 relative), or of the subnormals' (2^-10 scales)
        assert np.all(np.abs(v - xo) <= np.maximum(np.abs(xo) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-6))
    a, sa = fp8.quantize(bits, fp8.E5M2, e8m0, True, 0)
    b, sb = fp8.quantize(bits, fp8.E5M2, e8m0, True, 1)
    assert np.array_equal(a[:, :300].T, b[:, :200]) and np.array_equal(sa.T, sb)


def test_dropout_mask_rate_and_extremes():
    shape = (512, 513)
    assert dropout.keep(shape, 0.0, 1, 2).all()
    assert not dropout.keep(shape, 1.0, 1, 2).any()
    n = shape[0] * shape[1]
    for p in (0.1, 0.5, 0.9):
        q = 1 - dropout.threshold(p) / 65536  # binomial: five standard deviations
        assert abs(dropout.keep(shape, p, 7, 3).mean() - q) < 5 * np.sqrt(q * (1 - q) / n)
    # a stream of its own: not the stochastic rounding's bits, other seeds and offsets differ
    base = dropout.keep(shape, 0.5, 7, 3)
    assert (base != (philox.sr_bits(7, 3, 0, *shape) >= 32768)).mean() > 0.4
    for other in (dropout.keep(shape, 0.5, 8, 3), dropout.keep(shape, 0.5, 7, 4), dropout.keep(shape, 0.5, 7 + (1 << 32), 3)):
        assert 0.45 < (base != other).mean() < 0.55
    # element e alone decides: another shape of the same elements has the same mask
    assert np.array_equal(base.ravel(), dropout.keep((1, n), 0.5, 7, 3).ravel())


def test_dropout_values():
    x = np.float32([[1.0, np.nan, -2.0, np.inf]])
    m = np.array([[True, False, True, False]])
    assert dropout.dropout(x, m, 0.5).tolist() == [[2.0, 0.0, -4.0, 0.0]]
    assert dropout.dropout(x, m, 0.5, np.float32([[1, 1, 1, 1]])).tolist() == [[3.0, 1.0, -3.0, 1.0]]
    assert dropout.dropout(x, ~m & False, 1.0).tolist() == [[0.0] * 4]
