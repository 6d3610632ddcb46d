"""CPU tests of arguments that the experts' binding takes as well as refuses."""

import pytest
import torch

import fp4_block_scaled_amax_amd as lib
from test_binding_checks import Dev, raises
from test_experts_checks import dev, offs, quantized


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(Dev, "data_ptr", lambda self: 64)
    monkeypatch.setattr(lib.experts, "_launch", lambda where, device, stream, *args: seen.append((where, args)))
    return seen


def test_wgrad_takes_its_number_of_rows(calls):
    o, dw, a, b = offs(2), dev(2, 48, 64), quantized(48, 384), quantized(64, 384)
    for rows, taken in ((None, 128), (128, 128), (70, 70), (1, 1)):
        lib.gemm_grouped_wgrad(a, b, o, dw, rows=rows)
        where, args = calls.pop()
        assert where == "ue5m3fp4_gemm_grouped_wgrad" and args[7:9] == (2, taken)
    for rows in (0, 129, -1):
        raises(lambda: lib.gemm_grouped_wgrad(a, b, o, dw, rows=rows), "rows_padded")
    lib.gemm_grouped_wgrad(quantized(48, 256), quantized(64, 256), o, dw, rows=0)
    assert calls.pop()[1][7:9] == (2, 0)


def test_an_expert_counted_from_the_end():
    w = lib.empty_expert_weights(3, 10, 32, torch.ones(3))
    for g in (-1, -2, -3):
        q, want = w.expert(g), w.expert(3 + g)
        assert q.ts.numel() == 1 and q.ts.data_ptr() == want.ts.data_ptr()
        assert q.codes.data_ptr() == want.codes.data_ptr() and q.scales.data_ptr() == want.scales.data_ptr()
    for g in (3, -4):
        with pytest.raises(IndexError):
            w.expert(g)


def test_calls_run_with_their_device_current(monkeypatch):
    """The libraries launch on the current device: it is asked for, and changed for the call where it is another."""
    log = []

    class Current:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            log.append(("enter", self.d.index))

        def __exit__(self, *exc):
            log.append("exit")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", Current)
    launch = lambda *args: log.append(args) or 0  # noqa: E731
    lib.layer._enqueue(launch, "f", torch.device("cuda:1"), 5, 7)
    assert log == [(7, 5)]
    lib.layer._enqueue(launch, "f", torch.device("cuda:0"), 5, 7)
    assert log[1:] == [("enter", 0), (7, 5), "exit"]
