"""Dropout on the GPU: outputs bit for bit with the oracle (the mask from its
counters, one fp32 operation per step, one rounding), the amax by-product,
strides, the backward pass and offsets past 2^35 elements."""

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as lib
from oracle import dropout as oracle
from oracle import formats

from devhelpers import dev_scalar, host

pytestmark = pytest.mark.gpu

TYPES = ("bf16", "f32")
SEED = 0xDEADBEEF12345678


def values(shape, seed, kind):
    """(fp32 values of the type, device tensor)."""
    import torch

    v = np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)
    if kind == "bf16":
        bits = formats.f32_to_bf16_rne(v)
        return formats.bf16_to_f32(bits).reshape(shape), torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    return v, torch.from_numpy(v).cuda()


def rounded(v, kind):
    return formats.bf16_to_f32(formats.f32_to_bf16_rne(v)).reshape(v.shape) if kind == "bf16" else v


def empty(shape, kind):
    import torch

    return torch.full(shape, 7.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda")


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 5), (1, 8), (64, 64), (256, 257), (33, 1000), (1021, 24), (130, 4096)], ids=str)
def test_dropout_bit_exact(cuda_device, shape, kind, out, residual):
    x, xd = values(shape, 1, kind)
    r, rd = values(shape, 2, out) if residual else (None, None)
    for p, seed, offset in ((0.1, SEED, 5), (0.75, 3, 0xFFFFFFFF)):
        c, amax = empty(shape, out), dev_scalar(0.25)
        assert lib.dropout(xd, p, seed, offset, c, residual=rd, amax=amax) is c
        want = rounded(oracle.dropout(x, oracle.keep(shape, p, seed, offset), p, r), out)
        assert np.array_equal(host(c.float()), want)
        assert host(amax)[0] == max(np.float32(0.25), np.abs(want).max())
        lib.dropout(xd, p, seed, offset, c, residual=rd)  # without the amax
        assert np.array_equal(host(c.float()), want)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 1.5 * 2.0 ** -16, 1.0 - 2.0 ** -16, 1.0])
def test_extreme_probabilities(cuda_device, p):
    shape = (64, 1000)
    x, xd = values(shape, 3, "f32")
    r, rd = values(shape, 4, "f32")
    c = empty(shape, "f32")
    lib.dropout(xd, p, SEED, 1, c, residual=rd)
    assert np.array_equal(host(c), oracle.dropout(x, oracle.keep(shape, p, SEED, 1), p, r))
    if p == 1.0:
        assert np.array_equal(host(c), r)
    if p == 0.0:
        assert np.array_equal(host(c), x + r)


@pytest.mark.parametrize("cols,ldx,ldr,ldo", [(64, 72, 80, 88), (64, 64, 64, 96), (61, 64, 70, 65), (64, 65, 64, 64), (8, 8, 16, 8)])
@pytest.mark.parametrize("kind", TYPES)
def test_strided_rows(cuda_device, cols, ldx, ldr, ldo, kind):
    """Row strides of their own in each tensor; what lies beside the rows is left as it was."""
    rows = 77
    x, xd = values((rows, ldx), 5, kind)
    r, rd = values((rows, ldr), 6, "bf16")
    c = empty((rows, ldo), "bf16")
    lib.dropout(xd[:, :cols], 0.3, 11, 2, c[:, :cols], residual=rd[:, :cols])
    want = rounded(oracle.dropout(x[:, :cols], oracle.keep((rows, cols), 0.3, 11, 2), 0.3, r[:, :cols]), "bf16")
    assert np.array_equal(host(c[:, :cols].float()), want)
    assert (c[:, cols:] == 7).all()


def test_shapes_of_one_element_order_share_a_mask(cuda_device):
    import torch

    x, xd = values((6, 40, 16), 7, "bf16")
    a, b = torch.empty_like(xd), torch.empty((240, 16), dtype=torch.bfloat16, device="cuda")
    lib.dropout(xd, 0.4, 9, 9, a)
    lib.dropout(xd.view(240, 16), 0.4, 9, 9, b)
    assert torch.equal(a.view(240, 16), b)
    assert np.array_equal(host(a.float()).reshape(240, 16) != 0, (x.reshape(240, 16) != 0) & oracle.keep((240, 16), 0.4, 9, 9))
    with pytest.raises(ValueError):
        lib.dropout(xd[:, ::2], 0.4, 9, 9, a[:, ::2])  # neither contiguous nor a matrix


def test_in_place_and_dropped_nan(cuda_device):
    """out may be x or the residual; a dropped NaN or infinity contributes nothing, a kept one stays, the amax is NaN."""
    import torch

    shape = (50, 130)
    x, xd = values(shape, 8, "bf16")
    r, rd = values(shape, 9, "bf16")
    keep = oracle.keep(shape, 0.5, 1, 1)
    want = rounded(oracle.dropout(x, keep, 0.5, r), "bf16")
    for target in (xd.clone(), rd.clone()):
        into_x = torch.equal(target, xd)
        lib.dropout(target if into_x else xd, 0.5, 1, 1, target, residual=rd if into_x else target)
        assert np.array_equal(host(target.float()), want)
    drop = np.argwhere(~keep)
    for k, v in enumerate((float("nan"), float("inf"), float("-inf"))):
        xd[tuple(drop[k])] = v
    c, amax = empty(shape, "bf16"), dev_scalar(0)
    lib.dropout(xd, 0.5, 1, 1, c, residual=rd, amax=amax)
    assert np.array_equal(host(c.float()), want) and host(amax)[0] == np.abs(want).max()
    kept = np.argwhere(keep)
    xd[tuple(kept[0])] = float("-inf")
    lib.dropout(xd, 0.5, 1, 1, c, residual=rd, amax=amax)
    assert np.isneginf(host(c.float())[tuple(kept[0])]) and np.isinf(host(amax)[0])
    xd[tuple(kept[1])] = float("nan")
    lib.dropout(xd, 0.5, 1, 1, c, residual=rd, amax=amax)
    assert np.isnan(host(c.float())[tuple(kept[1])]) and np.isnan(host(amax)[0])


@pytest.mark.parametrize("kind", TYPES)
def test_backward_against_formula_and_differences(cuda_device, kind):
    import torch

    shape, p = (129, 515), 0.2
    g, gd = values(shape, 10, kind)
    dx, amax = empty(shape, kind), dev_scalar(0)
    lib.dropout_backward(gd, p, SEED, 77, dx, amax=amax)
    want = rounded(oracle.dropout(g, oracle.keep(shape, p, SEED, 77), p), kind)
    assert np.array_equal(host(dx.float()), want) and host(amax)[0] == np.abs(want).max()
    # the forward pass is linear in x: f(x + e) - f(x) = e * df/dx, exactly for small integers under scale 2
    x = torch.from_numpy(np.random.default_rng(1).integers(-8, 9, shape).astype(np.float32)).cuda()
    e = torch.from_numpy(np.random.default_rng(2).integers(-8, 9, shape).astype(np.float32)).cuda()
    one = torch.ones(shape, device="cuda")
    a, b, d = (torch.empty(shape, device="cuda") for _ in range(3))
    lib.dropout(x + e, 0.5, 4, 4, a, residual=x)
    lib.dropout(x, 0.5, 4, 4, b, residual=x)
    lib.dropout_backward(one, 0.5, 4, 4, d)
    assert torch.equal(a - b, e * d) and 0.45 < (d != 0).float().mean() < 0.55


def test_empty(cuda_device):
    import torch

    for shape in ((0,), (0, 8), (8, 0)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        amax = dev_scalar(0.5)
        lib.dropout(x, 0.5, 1, 1, torch.empty_like(x), amax=amax)
        assert host(amax)[0] == 0.5


def test_past_2_35_elements(cuda_device):
    """Call numbers past 2^32 use the counter's second word; offsets pass 2^36 bytes."""
    import torch

    rows, cols = 133120, 262144
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    lib.dropout(x, 0.5, SEED, 3, x)  # in place
    first = (1 << 35) // cols  # the row where call number 2^32 falls
    at = np.array([0, 1, first - 1, first, first + 1, rows - 1])
    got = host(x[torch.from_numpy(at).cuda()].float())
    assert np.array_equal(got, np.where(oracle.keep((rows, cols), 0.5, SEED, 3, rows=at), np.float32(2), np.float32(0)))
    for part in x.split(8192):
        assert bool(((part == 0) | (part == 2)).all())
