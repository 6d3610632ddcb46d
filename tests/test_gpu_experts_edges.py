"""GPU tests of the routed experts' operators at the edges of what they allow."""

import pytest

import fp4_block_scaled_amax_amd as lib
from devhelpers import dev_scalar
from test_gpu_experts_sizes import dev_i32, empty, rand_operand

pytestmark = pytest.mark.gpu

SCALES = [float("nan"), float("inf"), float("-inf"), 3e38]


@pytest.mark.parametrize("ts", SCALES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N", [(32, 48), (700, 704), (2100, 2000)])
def test_wgrad_of_no_rows_is_zero_under_any_scale(cuda_device, M, N, bf16, ts):
    E = 4
    a, b = rand_operand(M, lib.rows_padded(90, E), 1, ts), rand_operand(N, lib.rows_padded(90, E), 2)
    dw = empty((E, M, N), bf16)
    lib.gemm_grouped_wgrad(a, b, dev_i32([0, 0, 80, 80, 90]), dw)
    assert bool((dw[0] == 0).all()) and bool((dw[2] == 0).all())
    if ts != ts:
        assert bool(dw[1].isnan().all()) and bool(dw[3].isnan().all())
    lib.gemm_grouped_wgrad(b, a, dev_i32([0, 0, 0, 0, 0]), empty((E, N, M), bf16))


@pytest.mark.parametrize("ts", SCALES)
@pytest.mark.parametrize("rows,N", [(6, 9), (70, 9000)])
def test_products_of_no_elements_are_zero_under_any_scale(cuda_device, rows, N, ts):
    import torch

    u8 = dict(dtype=torch.uint8, device="cuda")
    none = lib.Quantized(torch.empty((rows, 0), **u8), torch.empty((rows, 0), **u8), dev_scalar(ts))
    o = dev_i32([0, 3, rows])
    for wts in (ts, 1.0):
        w = lib.empty_expert_weights(2, N, 0, dev_scalar(wts))
        for bf16 in (False, True):
            y, amax = empty((rows, N), bf16), dev_scalar(0.0)
            lib.gemm_grouped_fprop(none, w, o, y, amax=amax if bf16 else None)
            assert bool((y == 0).all()) and float(amax) == 0.0
            for n in (1, 3, rows):
                y = empty((n, N), bf16)
                lib.gemm_weight_only(torch.empty((n, 0), dtype=torch.bfloat16, device="cuda"), w.expert(1), y)
                assert bool((y == 0).all())


def test_wgrad_clamps_offsets_to_the_rows_it_is_given(cuda_device):
    """Offsets past the rows of the operands: quantizer and wgrad have to clamp them to the same number of rows, or wgrad
    reads columns that the quantizer never wrote."""
    import torch

    width, ts = 48, dev_scalar(0.01)
    for rows, raw, held in ((70, [0, 40, 70, 2 ** 31 - 1], [0, 40, 70, 70]), (130, [0, 100, 100, 1000], [0, 100, 100, 130]),
                            (129, [-5, 128, 500, 600], [0, 128, 129, 129]), (128, [0, 1, 90, 300], [0, 1, 90, 128])):
        P = lib.rows_padded(rows, 3)
        x = torch.randn((rows, width), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()

        def operand():
            u8 = dict(dtype=torch.uint8, device="cuda")
            return lib.Quantized(torch.full((width, P // 2), 0x77, **u8), torch.full((width, P // 16), 0xFF, **u8), ts)

        got, want = empty((3, width, width), False), empty((3, width, width), False)
        for o, dw in ((dev_i32(raw), got), (dev_i32(held), want)):
            q = operand()
            lib.quantize_grouped(x, o, ts, col=q)
            lib.gemm_grouped_wgrad(q, q, o, dw, rows=rows)
        assert bool(want.isfinite().all()) and torch.equal(got, want)
        q = operand()
        lib.quantize_grouped(x, dev_i32(held), ts, col=q)
        lib.gemm_grouped_wgrad(q, q, dev_i32(held), got)  # offsets inside the rows need no count of them
        assert torch.equal(got, want)
