"""Routed experts on streams: calls given a stream run on it, host threads with
streams of their own do not interfere, and captured graphs replay with other
inputs and offsets."""

import threading

import pytest

import fp4_block_scaled_amax_amd as lib
from devhelpers import dev_scalar
from test_gpu_experts_sizes import dev_i32, gen, rand_weights

pytestmark = pytest.mark.gpu


class Step:
    """A layer's calls on fixed buffers: quantize, the three products, a refresh of the scale, and a token's step."""

    def __init__(self, seed):
        import torch

        self.T, self.K, self.N, self.E = 400, 256, 384, 4
        T, K, N, E = self.T, self.K, self.N, self.E
        self.x = torch.randn((T, K), device="cuda", generator=gen(seed)).bfloat16()
        self.dy = torch.randn((T, N), device="cuda", generator=gen(seed + 1)).bfloat16()
        self.o = dev_i32([0, 100, 100, 333, 390])
        self.index = torch.randint(0, T, (T,), dtype=torch.int32, device="cuda", generator=gen(seed + 2))
        self.w, self.wt = rand_weights(E, N, K, seed + 3), rand_weights(E, K, N, seed + 4)
        self.ts, self.amax = dev_scalar(0.01), dev_scalar(0.0)
        P, u8 = lib.rows_padded(T, E), dict(dtype=torch.uint8, device="cuda")
        z = lambda r, c: lib.Quantized(torch.zeros((r, c // 2), **u8), torch.zeros((r, c // 16), **u8), self.ts)  # noqa: E731
        self.xr, self.xc, self.gr, self.gc = z(T, K), z(K, P), z(T, N), z(N, P)
        self.y, self.dx, self.dw, self.t, self.t1 = (torch.zeros(s, device="cuda", dtype=d) for s, d in (
            ((T, N), torch.bfloat16), ((T, K), torch.float32), ((E, N, K), torch.float32), ((40, N), torch.bfloat16),
            ((1, N), torch.float32)))

    def run(self, stream=None):
        s = dict(stream=stream)
        lib.quantize_grouped(self.x, self.o, self.ts, row=self.xr, col=self.xc, index=self.index, amax=self.amax, **s)
        lib.quantize_grouped(self.dy, self.o, self.ts, lib.SR, 11, 3, row=self.gr, col=self.gc, **s)
        lib.gemm_grouped_fprop(self.xr, self.w, self.o, self.y, **s)
        lib.gemm_grouped_dgrad(self.gr, self.wt, self.o, self.dx, **s)
        lib.gemm_grouped_wgrad(self.gc, self.xc, self.o, self.dw, **s)
        lib.gemm_weight_only(self.x[:40], self.w.expert(2), self.t, **s)
        lib.gemm_weight_only(self.x[:1], self.w.expert(1), self.t1, **s)

    def results(self):
        return [v.clone() for v in (self.xr.codes, self.xc.codes, self.xc.scales, self.gr.codes, self.gc.codes, self.amax,
                                    self.y, self.dx, self.dw, self.t, self.t1)]

    def clear(self):
        for q in (self.xr, self.xc, self.gr, self.gc):
            q.codes.zero_(), q.scales.zero_()
        for v in (self.y, self.dx, self.dw, self.t, self.t1, self.amax):
            v.zero_()


def same(a, b):
    import torch

    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_given_stream_orders_the_work(cuda_device):
    """Inputs that arrive on a stream are seen by calls given that stream, while another one is current."""
    import torch

    step = Step(20)
    step.run()
    want = step.results()
    s, x, dy = torch.cuda.Stream(), step.x.clone(), step.dy.clone()
    step.clear()
    step.x.zero_(), step.dy.zero_()
    torch.cuda.synchronize()
    busy = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):  # milliseconds of work ahead of the inputs
            busy = busy @ busy * 1e-3
        step.x.copy_(x), step.dy.copy_(dy)
    step.run(stream=s)
    s.synchronize()
    assert same(step.results(), want)


def test_threads_on_their_own_streams(cuda_device):
    import torch

    steps = [Step(30), Step(40), Step(45)]
    want = []
    for s in steps:
        s.run()
        want.append(s.results())
    torch.cuda.synchronize()
    good, errors = [], []

    def work(step, ref):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    step.clear()
                    step.run()
                    good.append(same(step.results(), ref))
        except Exception as e:  # reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(steps, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(100)
    assert not errors and len(good) == 60 and all(good)


def test_captured_steps_replay(cuda_device):
    """Two graphs of the calls, replayed in turn with other inputs, other offsets and eager calls between."""
    import torch

    steps = [Step(50), Step(60)]
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    splits = [[0, 100, 100, 333, 390], [5, 5, 300, 301, 400], [0, 0, 0, 0, 0], [0, 400, 400, 400, 400]]
    for r, split in enumerate(splits):
        want = []
        for i, s in enumerate(steps):
            s.x.copy_(torch.randn(s.x.shape, device="cuda", generator=gen(100 * r + i)))
            s.o.copy_(dev_i32(split))
            s.clear()
            s.run()  # eager
            want.append(s.results())
            s.clear()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, ref in zip(steps, want):
            assert same(s.results(), ref), f"replay {r}"
