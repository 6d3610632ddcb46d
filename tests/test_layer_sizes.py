"""CPU tests of the sizes that the layer operators take: what the C ABI admits
(the checks come before any HIP call, in the order range, pointers) and the
rows, columns and strides that the binding hands down for tensors of any
dimension."""

import pytest
import torch

import fp4_block_scaled_amax_amd as lib
from fp4_block_scaled_amax_amd import layer
from test_binding_checks import Dev
from test_layer_checks import EINVAL, ERANGE, L, P, dr  # noqa: F401  (L: the fixture)


def test_dropout_columns_have_no_limit_of_their_own(L):  # noqa: F811
    """In range: the missing x is what is refused."""
    for rows, cols in ((8, 1 << 31), (1, (1 << 40) - 1), (1, (1 << 32) + 8), (511, 1 << 31)):
        assert dr(L, rows=rows, cols=cols, ldx=cols, ldo=cols, x=None) == EINVAL
        assert dr(L, rows=rows, cols=cols, ldx=cols, ldo=cols, r=P, ldr=cols, x=None) == EINVAL
    for rows, cols in ((512, 1 << 31), (1, 1 << 40), (2, 1 << 39), (1, (1 << 63) - 1)):
        assert dr(L, rows=rows, cols=cols, ldx=cols, ldo=cols, x=None) == ERANGE
    assert dr(L, rows=512, cols=32, ldx=32, ldo=32, r=P, ldr=1 << 31, x=None) == ERANGE


class Placed(Dev):
    """A stand-in of any size (a meta tensor) that has an address; nothing is launched in these tests."""

    def data_ptr(self):
        return P


@pytest.mark.parametrize("shape,handed", [
    ((2, 8192, 131080), (1, 2 * 8192 * 131080)), (((1 << 31) + 24,), (1, (1 << 31) + 24)), ((), (1, 1)),
    ((4, 5, 0), (1, 0)), ((0, 5, 8), (1, 0)), ((7, 9), (7, 9)), ((7, 0), (7, 0)), ((2, 3, 4, 5), (1, 120))], ids=str)
def test_dropout_hands_down_rows_columns_and_strides(monkeypatch, shape, handed):
    seen = []
    monkeypatch.setattr(layer, "_launch", lambda where, device, stream, *args: seen.append((where, args)))
    x, out, res = (Placed(torch.empty(shape, dtype=torch.bfloat16, device="meta")) for _ in range(3))
    assert lib.dropout(x, 0.5, 3, 4, out, residual=res) is out
    lib.dropout_backward(x, 0.5, 3, 4, out)
    rows, cols = handed
    assert seen[0] == ("ue5m3fp4_dropout", (P, 0, cols, P, cols, P, 0, cols, rows, cols, 0.5, 3, 4, None))
    assert seen[1] == ("ue5m3fp4_dropout_backward", (P, 0, cols, P, 0, cols, rows, cols, 0.5, 3, 4, None))
