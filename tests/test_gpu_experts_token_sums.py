"""GPU tests of the weight-only product where its sums are longest, and where the
tokens are smallest, at the library's bar 1e-5 * |ts| * sum |a b|: sums of 256 matrix
instructions, 2^-16 = 1.5e-5 at most and half of that on average over a growing sum,
are joined to longer ones.
"""

import pytest

import fp4_block_scaled_amax_amd as lib
from test_gpu_experts_sizes import empty, gen, rand_operand, values
from test_gpu_experts_sums import KINDS, check_sampled, long_operand, products, sampled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 3, 16, 33])
@pytest.mark.parametrize("N,K", [(40, (1 << 23) + 528), (8, 1 << 23), (16400, (1 << 18) + 512)])
def test_weight_only_long_contractions(cuda_device, rows, N, K, kind):
    import torch

    w = long_operand(N, K, 7, kind)
    x = torch.randn((rows, K), device="cuda", generator=gen(8)).bfloat16()
    x = torch.full_like(x, 1.2578125) if kind == "equal" else x.abs() if kind == "positive" else x
    out = empty((rows, N), False)
    lib.gemm_weight_only(x, w, out)
    ib = sampled(N)
    ref = torch.zeros((rows, len(ib)), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    for c in range(0, K, 1 << 19):
        v = values(lib.Quantized(w.codes[ib, c // 2:c // 2 + (1 << 18)], w.scales[ib, c // 16:c // 16 + (1 << 15)], w.ts))
        r, s = products(x[:, c:c + (1 << 19)].double(), v)
        ref += r
        bound += s
    check_sampled(out, list(range(rows)), ib, ref, 1e-5 * bound)


@pytest.mark.parametrize("rows", [1, 2, 4, 16, 32, 64])
@pytest.mark.parametrize("K", [16, 512, 528, 1152])
def test_weight_only_smallest_tokens(cuda_device, rows, K):
    """Tokens of bf16's smallest normal numbers, 2^-126 to 2^-118, times large weights: results are normal numbers, and
    every form has them."""
    import torch

    N = 40
    w = rand_operand(N, K, 9)
    w.scales.copy_(torch.randint(0xC0, 0xFE, w.scales.shape, dtype=torch.uint8, device="cuda", generator=gen(10)))
    x = torch.rand((rows, K), device="cuda", generator=gen(11)) + 1.0
    x = x * torch.exp2(-126.0 + torch.randint(0, 8, x.shape, device="cuda", generator=gen(12)))
    x = (x * torch.where(torch.rand(x.shape, device="cuda", generator=gen(13)) < 0.5, -1.0, 1.0)).bfloat16()
    assert bool((x.abs() >= 2.0 ** -126).all())
    out = empty((rows, N), False)
    lib.gemm_weight_only(x, w, out)
    wv, xv = values(w), x.double()
    ref, lim = xv @ wv.t().contiguous(), 1e-5 * (xv.abs() @ wv.abs().t().contiguous())
    assert bool(((out.double() - ref).abs() <= lim).all()), float(((out.double() - ref).abs() / lim * 1e-5).max())
