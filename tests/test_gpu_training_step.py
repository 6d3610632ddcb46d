"""The layer operators together, as a training step uses them: an 8-bit linear,
dropout joined to the residual stream with the amax that refreshes the FP4
tensor scale, the FP4 linear behind it, and the way back -- eagerly, on a side
stream, captured into a graph and replayed, and from two threads at once.

(The file's name places it behind test_gpu_streams.py: the control there needs
its side stream on another hardware queue than the default stream's, and the
streams that are taken from torch's pool here would move it.)"""

import threading

import numpy as np
import pytest

import fp4_block_scaled_amax_amd as lib
from oracle import dropout as drop_oracle
from oracle import formats, fp8, quantize, tensor_scale
from workloads import random_bf16

from devhelpers import dev_bf16, dev_scalar, host

pytestmark = pytest.mark.gpu

T, I, O, P, SEED = 200, 272, 384, 0.25, 99


class Step:
    """Buffers and one pass: h = residual + dropout(x W8^T), y = fp4(h) W4^T, and the gradients of the 8-bit linear."""

    def __init__(self, seed):
        import torch

        self.bits = {"x": random_bf16((T, I), seed, "heavy"), "w8": random_bf16((O, I), seed + 1), "res": random_bf16((T, O), seed + 2),
                     "w4": random_bf16((64, O), seed + 3), "g": random_bf16((T, O), seed + 4, "gradient")}
        b16 = {k: dev_bf16(v).view(torch.bfloat16) for k, v in self.bits.items()}
        self.b16 = b16
        e = lib.empty_quantized_fp8
        self.q = {"xr": e(T, I), "xc": e(I, T), "wr": e(O, I, tile=True), "wc": e(I, O, tile=True),
                  "gr": e(T, O, lib.E5M2), "gc": e(O, T, lib.E5M2)}
        self.z = torch.empty((T, O), dtype=torch.float32, device="cuda")
        self.h = torch.empty((T, O), dtype=torch.bfloat16, device="cuda")
        self.dz = torch.empty_like(self.h)
        self.amax, self.gmax = dev_scalar(0), dev_scalar(0)
        self.ts, self.wts = dev_scalar(1), dev_scalar(1e-4)
        self.h4, self.w4 = lib.empty_quantized(T, O, self.ts), lib.empty_quantized(64, O, self.wts)
        self.y = torch.empty((T, 64), dtype=torch.float32, device="cuda")
        self.dx = torch.empty((T, I), dtype=torch.bfloat16, device="cuda")
        self.dw = torch.empty((O, I), dtype=torch.float32, device="cuda")

    def run(self, stream=None):
        q, s = self.q, dict(stream=stream)
        lib.quantize_fp8(self.b16["x"], row=q["xr"], col=q["xc"], **s)
        lib.quantize_fp8(self.b16["w8"], row=q["wr"], col=q["wc"], **s)
        lib.gemm_fp8_fprop(q["xr"], q["wr"], self.z, **s)
        lib.dropout(self.z, P, SEED, 1, self.h, residual=self.b16["res"], amax=self.amax, **s)
        lib.update_tensor_scale(self.amax, self.ts, 0, 1, **s)
        lib.quantize_blockscale(self.h, self.ts, row=self.h4, **s)
        lib.quantize_blockscale(self.b16["w4"], self.wts, row=self.w4, **s)
        lib.gemm_fprop(self.h4, self.w4, self.y, **s)
        lib.dropout_backward(self.b16["g"], P, SEED, 1, self.dz, amax=self.gmax, **s)
        lib.quantize_fp8(self.dz, row=q["gr"], col=q["gc"], **s)
        lib.gemm_fp8_dgrad(q["gr"], q["wc"], self.dx, **s)
        lib.gemm_fp8_wgrad(q["gc"], q["xc"], self.dw, **s)

    def reset(self):
        for t in (self.z, self.h, self.dz, self.y, self.dx, self.dw):
            t.fill_(-3)
        for v in self.q.values():
            v.codes.fill_(0x5A)
            v.scales.fill_(0x5A)
        self.amax.fill_(0)
        self.gmax.fill_(0)
        self.ts.fill_(1)

    def results(self):
        return {k: getattr(self, k).clone() for k in ("z", "h", "dz", "y", "dx", "dw", "ts", "gmax")}


def same(a, b):
    import torch

    return all(torch.equal(a[k], b[k]) for k in a)


def test_step_against_the_oracles(cuda_device):
    s = Step(1)
    s.run()
    ops = {k: fp8.operand(*fp8.quantize(s.bits[b], fp8.E4M3, False, t, 0), fp8.E4M3, t) for k, b, t in (("x", "x", False), ("w", "w8", True))}
    z = host(s.z)
    ref, sab = fp8.gemm_nt(ops["x"], ops["w"])
    assert np.all(np.abs(z - ref) <= 1e-5 * sab)
    # from the GPU's own z on, every step is bit exact
    h = drop_oracle.dropout(z, drop_oracle.keep((T, O), P, SEED, 1), P, formats.bf16_to_f32(s.bits["res"]).reshape(T, O))
    hb = formats.f32_to_bf16_rne(h)
    assert np.array_equal(host(s.h.float()), formats.bf16_to_f32(hb).reshape(T, O))
    _, ts = tensor_scale.update_tensor_scale(quantize.tensor_amax(hb.reshape(T, O)), np.float32(1), 0, 1)
    assert host(s.ts)[0] == ts
    codes, scales = quantize.quantize_blockscale(hb.reshape(T, O), ts)
    assert np.array_equal(host(s.h4.codes), codes) and np.array_equal(host(s.h4.scales), scales)
    dz = drop_oracle.dropout(formats.bf16_to_f32(s.bits["g"]).reshape(T, O), drop_oracle.keep((T, O), P, SEED, 1), P)
    db = formats.f32_to_bf16_rne(dz).reshape(T, O)
    assert np.array_equal(host(s.dz.float()), formats.bf16_to_f32(db).reshape(T, O))
    g = fp8.operand(*fp8.quantize(db, fp8.E5M2, False, False, 1), fp8.E5M2, False)
    x = fp8.operand(*fp8.quantize(s.bits["x"], fp8.E4M3, False, False, 1), fp8.E4M3, False)
    ref, sab = fp8.gemm_nt(g, x)
    assert np.all(np.abs(host(s.dw) - ref) <= 1e-5 * sab)


def test_side_stream_and_graph(cuda_device):
    import torch

    s = Step(2)
    s.run()
    torch.cuda.synchronize()
    eager = s.results()

    side = torch.cuda.Stream()
    s.reset()
    torch.cuda.synchronize()
    s.run(side)
    side.synchronize()
    assert same(eager, s.results())

    s.reset()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):  # torch's current stream
        s.run()
    side.synchronize()
    assert same(eager, s.results())

    g = torch.cuda.CUDAGraph()
    other = Step(3)
    with torch.cuda.graph(g):
        s.run()
        other.run()
    for _ in range(3):
        s.reset()
        other.reset()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(eager, s.results())
        torch.randn(512, 512, device="cuda").sum().item()  # eager work between the replays
        got = other.results()
        other.reset()
        other.run()
        torch.cuda.synchronize()
        assert same(got, other.results())


def test_two_threads_on_their_own_streams(cuda_device):
    import torch

    steps = [Step(10), Step(20)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
        s.reset()
    torch.cuda.synchronize()
    errors = []

    def work(s, ref):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                s.amax.fill_(0)
                torch.cuda.synchronize()
                s.run(stream)
                stream.synchronize()
                if not same(ref, s.results()):
                    errors.append("results differ")
        except Exception as e:  # reported by the assertion below
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(steps, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:3]


def test_stream_of_another_device_is_refused(cuda_device):
    import torch

    s = Step(4)

    class Elsewhere:
        device = torch.device("cuda:7")
        cuda_stream = 0

    with pytest.raises(ValueError, match="stream belongs to"):
        lib.quantize_fp8(s.b16["x"], row=s.q["xr"], stream=Elsewhere())


def test_readme_layer_example(cuda_device):
    """The README's second example runs as written behind the first; its GEMMs agree with fp64 products of the
    operands they were given, its dropout with the oracle's mask."""
    import os

    import torch

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    ns = {}
    for block in text.split("```python\n")[1:3]:
        exec(compile(block[:block.index("```")], "README.md", "exec"), ns)
    torch.cuda.synchronize()

    def values(q):
        return fp8.operand(host(q.codes), host(q.scales), q.fmt, q.tile)

    rows = slice(0, 64)
    X, W, G = ns["X8"], ns["W8"], ns["G8"]
    for out, a, b, rel in ((ns["y"], X[0], W[0], 1e-5), (ns["dx16"], G[0], W[1], 2.0 ** -8), (ns["dw"], G[1], X[1], 1e-5)):
        ref, _ = fp8.gemm_nt(values(a)[rows], values(b))
        got = host(out[rows].double())
        assert np.linalg.norm(got - ref) <= rel * np.linalg.norm(ref)
    keep = drop_oracle.keep(tuple(ns["h"].shape), 0.1, 1234, 0)
    want = formats.f32_to_bf16_rne(drop_oracle.dropout(host(ns["y"]), keep, 0.1))
    assert np.array_equal(host(ns["h"].float()), formats.bf16_to_f32(want).reshape(keep.shape))
    assert host(ns["amax"])[0] == np.abs(formats.bf16_to_f32(want)).max()
    dz = formats.f32_to_bf16_rne(drop_oracle.dropout(host(ns["dy"].float()), keep, 0.1))
    assert np.array_equal(host(ns["dz"].float()), formats.bf16_to_f32(dz).reshape(keep.shape))
