"""The largest sizes of the layer operators on the GPU: more workgroups than one
launch holds (HIP takes fewer than 2^32 threads per grid dimension, and starts
their number modulo 2^32 beyond), and contiguous tensors of any dimension past
2^31 elements."""

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as lib
from oracle import dropout as oracle
from oracle import formats, fp8

from devhelpers import host

pytestmark = pytest.mark.gpu

TALL = (1 << 29) + 70  # rows of C whose 64 x 64 tiles of 512 threads pass 2^32 threads


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(TALL, 1), (1, TALL)], ids=["tall", "wide"])
def test_gemm_empty_sum_of_many_tiles(cuda_device, shape, out):
    import torch

    c = torch.full(shape, 3.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    lib.gemm_fp8_nt(lib.empty_quantized_fp8(shape[0], 0), lib.empty_quantized_fp8(shape[1], 0), c)
    assert not bool(c.any())


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gemm_many_tiles(cuda_device, out):
    """One code per row, one column: C(i) is row i's value times its tile's scale, whichever launch holds it."""
    import torch

    codes = torch.zeros((TALL, 128), dtype=torch.uint8, device="cuda")  # 64 GiB
    i = torch.arange(TALL, device="cuda", dtype=torch.int32)
    codes[:, 0] = (i % 7).to(torch.uint8) + 0x38  # 1, 1.125 ... 1.75
    tiles = -(-TALL // 128)
    scales = (1 << (torch.arange(tiles, device="cuda") % 5)).float()[None]
    a = lib.Fp8Quantized(codes, scales, 1, lib.E4M3, True)
    b = lib.empty_quantized_fp8(1, 1)
    b.codes.zero_()
    b.codes[0, 0] = 0x40  # 2
    b.scales.fill_(0.5)
    c = torch.full((TALL, 1), -1.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    lib.gemm_fp8_nt(a, b, c)
    del a, codes
    want = (1 + (i % 7).float() / 8) * (1 << (i // 128 % 5)).float()
    assert torch.equal(c[:, 0].float(), want)


def test_dropout_of_many_units(cuda_device):
    """2^37 elements and more, in place: 2^24 workgroups of 256 threads."""
    import torch

    rows, cols = (1 << 19) + 3, 1 << 18
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < rows * cols * 2 + (4 << 30):
        pytest.skip("a bf16 tensor of 2^37 elements does not fit this GPU")
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for part in x.split(8192):
        part.fill_(1.0)
    lib.dropout(x, 0.5, 0xDEADBEEF12345678, 3, x)
    at = np.array([0, (1 << 17) - 1, 1 << 17, (1 << 19) - 1, 1 << 19, rows - 1])
    got = host(x[torch.from_numpy(at).cuda()].float())
    assert np.array_equal(got, np.where(oracle.keep((rows, cols), 0.5, 0xDEADBEEF12345678, 3, rows=at), np.float32(2), np.float32(0)))
    for part in x.split(2048):
        assert not bool((part == 1).any())
    del x, part
    torch.cuda.empty_cache()


def test_transposed_quantization_of_many_tiles(cuda_device):
    """One column of 2^31 - 1 rows: 2^24 tiles of 256 threads."""
    import torch

    R, period = (1 << 31) - 1, 128 * 5
    v = np.random.default_rng(1).standard_normal(period, dtype=np.float32)
    bits = formats.f32_to_bf16_rne(v).reshape(period, 1)
    one = torch.from_numpy(bits.view(np.int16)).cuda()
    x = one.repeat(-(-R // period), 1)[:R].contiguous().view(torch.bfloat16)
    q = lib.empty_quantized_fp8(1, R)
    q.codes.fill_(0x5A)
    q.scales.fill_(-1)
    lib.quantize_fp8(x, col=q)
    codes, scales = fp8.quantize(bits, lib.E4M3, orientation=1)
    whole = R // period * period
    want = torch.from_numpy(codes).cuda().reshape(-1)
    assert all(bool((part.view(-1, period) == want).all()) for part in q.codes[0, :whole].split(period << 15))
    assert bool((q.scales[:whole // 128, 0].view(-1, 5) == torch.from_numpy(scales).cuda().view(-1)).all())
    # the ragged end, its zero padding included
    codes, scales = fp8.quantize(bits[:R - whole], lib.E4M3, orientation=1)
    assert np.array_equal(host(q.codes[:, whole:]), codes)
    assert np.array_equal(host(q.scales[whole // 128:]), scales)


@pytest.mark.parametrize("shape", [(2, 8192, 131080), ((1 << 31) + 24,)], ids=["3d", "1d"])
def test_dropout_of_contiguous_tensors_past_2_31_elements(cuda_device, shape):
    """The mask of element e is that of the tensor's matrix view."""
    import torch

    cols = 131080 if len(shape) == 3 else 8
    x = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    lib.dropout(x, 0.5, 7, 9, y, residual=x)
    lib.dropout_backward(x, 0.5, 7, 9, x)
    y, x = y.view(-1, cols), x.view(-1, cols)
    assert torch.equal(y, x + 1)  # 3 and 2 where kept, 1 and 0 where dropped
    rows = np.array([0, 1, (1 << 31) // cols - 1, (1 << 31) // cols, x.shape[0] - 1])
    keep = oracle.keep(tuple(x.shape), 0.5, 7, 9, rows=rows)
    assert np.array_equal(host(x[torch.from_numpy(rows).cuda()].float()) != 0, keep)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1480, 2900], ids=["128", "256"])
def test_gemm_longest_contraction(cuda_device, n, out):
    """K of 2^24 - 1: code offsets within a tile of 128 (256) rows pass 2^31 (come near 2^32).  +-1 in five
    patterns a side: every sum is an integer of at most 2^24, exact in fp32."""
    import torch

    K, D = (1 << 24) - 1, 5
    g = torch.Generator(device="cuda").manual_seed(n)
    pats = [torch.randint(0, 2, (D, K + 1), generator=g, device="cuda", dtype=torch.int8) * 2 - 1 for _ in range(2)]
    ref = torch.zeros((D, D), dtype=torch.float64, device="cuda")
    ops, i = [], torch.arange(n, device="cuda") % D
    for p in pats:
        p[:, K:] = 0
        codes = torch.where(p == 0, 0, torch.where(p > 0, 0x38, 0xB8)).to(torch.uint8)
        tile = not ops  # A under tile scales, B under 1-D ones
        scales = torch.ones(((K + 1) // 128, -(-n // 128) if tile else n), device="cuda")
        ops.append(lib.Fp8Quantized(codes[i], scales, K, lib.E4M3, tile))
    for x, y in zip(pats[0].split(1 << 20, dim=1), pats[1].split(1 << 20, dim=1)):
        ref += torch.mm(x.double(), y.double().t().contiguous())
    c = torch.full((n, n), float("nan"), dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    lib.gemm_fp8_nt(*ops, c)
    assert torch.equal(c, ref[i][:, i].to(c.dtype))
    del ops
    torch.cuda.empty_cache()
