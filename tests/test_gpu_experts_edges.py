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
