"""The 8-bit block-128 linear and the counter-based dropout: cases, plain forms and calls.

Operators:
  * quantize: a bf16 tensor to 8-bit codes (E4M3 or E5M2) with one scale per 128 elements of a row (1-D blocks) or
    per 128 x 128 tile, as the row-wise operand (blocked along the columns) and / or the transposed operand (blocked
    along the rows) of the GEMMs;
  * product: fprop, dgrad and wgrad of a linear layer on such operands;
  * dropout: out = residual + dropout(x) with a mask from Philox4x32-10 that is never stored, and its backward pass.

Layouts.  An R x C operand: codes [R][ceil(C / 128) * 128] (zero beyond C); scales [ceil(C / 128)][R], or
[ceil(C / 128)][ceil(R / 128)] for tiles, fp32 or E8M0 bytes (2^(c - 127)).
"""

import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def up(n, k=128):
    return (n + k - 1) // k * k


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the activations of an attention projection, both operands from one read
        dict(name="quantize activations", op="quantize", rows=8192, cols=4096, fmt="e4m3", pow2=False, tile=False,
             row=True, col=True, kind="activation"),
        # the gradient of the wide FFN output, in the format with the larger range
        dict(name="quantize gradient", op="quantize", rows=8192, cols=16384, fmt="e5m2", pow2=False, tile=False,
             row=True, col=True, kind="gradient"),
        # a weight once per step: one scale per tile serves both operands, powers of two
        dict(name="quantize weight tiles", op="quantize", rows=16384, cols=4096, fmt="e4m3", pow2=True, tile=True,
             row=True, col=True, kind="weight"),
        # a short ragged batch before fprop: latency
        dict(name="quantize few tokens", op="quantize", rows=17, cols=4104, fmt="e4m3", pow2=False, tile=False,
             row=True, col=False, kind="activation"),
        # up projection, forward
        dict(name="fprop up", op="product", role="fprop", tokens=8192, inputs=4096, outputs=16384, fmt="e4m3",
             pow2=False, tile=True, out="bf16"),
        # up projection, input gradient: E5M2 times E4M3 under power-of-two scales
        dict(name="dgrad up", op="product", role="dgrad", tokens=8192, inputs=4096, outputs=16384, fmt="e5m2",
             pow2=True, tile=True, out="bf16"),
        # attention projection, weight gradient: 1-D scales on both sides, fp32 result
        dict(name="wgrad projection", op="product", role="wgrad", tokens=8192, inputs=4096, outputs=4096, fmt="e4m3",
             pow2=False, tile=False, out="f32"),
        # a ragged micro-batch through a layer of odd sizes
        dict(name="fprop ragged", op="product", role="fprop", tokens=1531, inputs=2056, outputs=1305, fmt="e4m3",
             pow2=False, tile=True, out="f32"),
        # one token at a time through the up projection (evaluation by generation)
        dict(name="fprop one token", op="product", role="fprop", tokens=1, inputs=4096, outputs=16384, fmt="e4m3",
             pow2=False, tile=True, out="bf16"),
        # a tiny layer's activations: latency
        dict(name="dropout small", op="dropout", rows=256, cols=257, x="bf16", out="bf16", residual=False, p=0.1,
             backward=False),
        # an fp32 GEMM output joined to the bf16 residual stream, with the amax the next quantizer scales by
        dict(name="dropout residual", op="dropout", rows=8192, cols=4096, x="f32", out="bf16", residual=True, p=0.1,
             backward=False),
        # the gradient of the wide FFN activation
        dict(name="dropout backward", op="dropout", rows=8192, cols=16384, x="bf16", out="bf16", residual=False,
             p=0.25, backward=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "dropout"])
    if op == "quantize":
        rows = _log(rng, 1, 16384)
        cols = _log(rng, 16, min(16384, 8192 * 16384 // rows))
        outputs = rng.choice(["row", "col", "both", "both"])
        return dict(op=op, rows=rows, cols=cols, fmt=rng.choice(["e4m3", "e5m2"]), pow2=rng.random() < 0.5,
                    tile=rng.random() < 0.4, row=outputs != "col", col=outputs != "row",
                    kind=rng.choice(["activation", "weight", "gradient"]))
    if op == "product":
        role = rng.choice(["fprop", "dgrad", "wgrad"])
        a, b = _log(rng, 64, 16384), _log(rng, 64, 16384)
        t = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 16384 // (a * b))))
        return dict(op=op, role=role, tokens=t, inputs=a, outputs=b, fmt=rng.choice(["e4m3", "e5m2"]),
                    pow2=rng.random() < 0.4, tile=role != "wgrad" and rng.random() < 0.7,
                    out=rng.choice(["bf16", "f32"]))
    backward = rng.random() < 0.4
    return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 1, 16384), x=rng.choice(["bf16", "f32"]),
                out=rng.choice(["bf16", "f32"]), residual=not backward and rng.random() < 0.6,
                p=round(rng.uniform(0.02, 0.6), 3), backward=backward)


# ------------------------------------------------------------------ inputs --

def _values(kind, rows, cols, gen):
    z = torch.randn((rows, cols), generator=gen, device="cuda")
    if kind == "activation":  # heavy tails and a few outlier columns
        z *= torch.exp(0.5 * torch.randn((1, cols), generator=gen, device="cuda"))
        at = torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device="cuda")
        z[:, at] *= 30.0
    elif kind == "weight":
        z *= 0.02
    else:  # gradients: a magnitude of its own for each token
        z *= 1e-3 * torch.exp(torch.randn((rows, 1), generator=gen, device="cuda"))
    return z.to(torch.bfloat16)


def _quantized(x, fmt, pow2, tile):
    """(codes, scales) of x blocked along its columns, by the definition, in 32 bits."""
    R, C = x.shape
    g = 128 if tile else 1
    Cp, Rp = up(C), up(R, g)
    w = torch.zeros((Rp, Cp), dtype=torch.float32, device=x.device)
    w[:R, :C] = x.float()
    w = w.view(Rp // g, g, Cp // 128, 128)
    a = w.abs().amax(dim=(1, 3))
    largest = torch.tensor(LARGEST[fmt], dtype=torch.float32, device=x.device)
    s = a / largest
    if pow2:
        mantissa, e = torch.frexp(s)                      # s = mantissa * 2^e, mantissa in [0.5, 1)
        e = torch.where(mantissa == 0.5, e - 1, e)
        e = torch.where(s == 0, torch.full_like(e, -127), e).clamp(min=-127)
        s = torch.ldexp(torch.ones_like(s, dtype=torch.float64), e).float()
        kept = (e + 127).to(torch.uint8)
    else:
        s = s.clamp(min=2.0 ** -126)
        kept = s
    v = w * (1.0 / s)[:, None, :, None]
    codes = v.clamp(-LARGEST[fmt], LARGEST[fmt]).to(F8[fmt]).view(torch.uint8).view(Rp, Cp)[:R].contiguous()
    return codes, kept.t().contiguous()


def _empty(rows, cols, pow2, tile):
    return (torch.empty((rows, up(cols)), dtype=torch.uint8, device="cuda"),
            torch.empty((up(cols) // 128, up(rows) // 128 if tile else rows),
                        dtype=torch.uint8 if pow2 else torch.float32, device="cuda"))


def _mnk(case):
    t, i, o = case["tokens"], case["inputs"], case["outputs"]
    return {"fprop": (t, o, i), "dgrad": (t, i, o), "wgrad": (o, i, t)}[case["role"]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case, seed=seed)
    if case["op"] == "quantize":
        R, C = case["rows"], case["cols"]
        s["x"] = _values(case["kind"], R, C, gen)
        s["row_out"] = _empty(R, C, case["pow2"], case["tile"]) if case["row"] else None
        s["col_out"] = _empty(C, R, case["pow2"], case["tile"]) if case["col"] else None
    elif case["op"] == "product":
        M, N, K = _mnk(case)
        s["K"] = K
        a_kind, b_kind = {"fprop": ("activation", "weight"), "dgrad": ("gradient", "weight"),
                          "wgrad": ("gradient", "activation")}[case["role"]]
        s["a"] = _quantized(_values(a_kind, M, K, gen), case["fmt"], case["pow2"], False)
        s["b"] = _quantized(_values(b_kind, N, K, gen), "e4m3", case["pow2"], case["tile"])
        s["c"] = torch.empty((M, N), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device="cuda")
    else:
        shape, types = (case["rows"], case["cols"]), {"bf16": torch.bfloat16, "f32": torch.float32}
        s["in"] = (torch.randn(shape, generator=gen, device="cuda") * (1e-3 if case["backward"] else 1.0)).to(types[case["x"]])
        s["res"] = torch.randn(shape, generator=gen, device="cuda").to(types[case["out"]]) if case["residual"] else None
        s["c"] = torch.empty(shape, dtype=types[case["out"]], device="cuda")
        s["amax"] = torch.zeros(1, dtype=torch.float32, device="cuda")
        s["key"], s["step"] = 0x9E3779B97F4A7C15 ^ (seed * 0x2545F491), 7 + seed % 1000
    return s


# -------------------------------------------------------------- plain forms --

def _scale_values(scales):
    return torch.ldexp(torch.ones((), dtype=torch.float64, device=scales.device),
                       scales.to(torch.int32) - 127).float() if scales.dtype == torch.uint8 else scales


def _operand_values(q, fmt, tile):
    codes, scales = q
    s = _scale_values(scales)
    if tile:
        s = s.repeat_interleave(128, dim=1)[:, :codes.shape[0]]
    v = codes.view(F8[fmt]).to(torch.float32).view(codes.shape[0], -1, 128)
    return (v * s.t().unsqueeze(2)).view(codes.shape)


M32 = 0xFFFFFFFF


def _round(c, k):
    """One Philox round; the products wrap in 64 bits, their halves are masked out."""
    p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
    return [((p1 >> 32) & M32) ^ c[1] ^ k[0], p1 & M32, ((p0 >> 32) & M32) ^ c[3] ^ k[1], p0 & M32]


def _random16(n, key, offset):
    """The 16 random bits of elements 0 .. n - 1."""
    call = torch.arange((n + 7) // 8, dtype=torch.int64, device="cuda")
    c = [call & M32, call >> 32, torch.full_like(call, offset), torch.full_like(call, 2)]
    k0, k1 = key & M32, (key >> 32) & M32
    for r in range(10):
        c = _round(c, ((k0 + r * 0x9E3779B9) & M32, (k1 + r * 0xBB67AE85) & M32))
    return torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], dim=1).view(-1)[:n]


def _plain_dropout(s):
    t = round(65536 * s["p"])
    x = s["in"].float()
    keep = (_random16(x.numel(), s["key"], s["step"]) >= t).view(x.shape)
    scale = torch.tensor(65536.0 / (65536 - t), dtype=torch.float32, device="cuda")
    y = torch.where(keep, x * scale, torch.zeros_like(x))
    if s["res"] is not None:
        y = s["res"].float() + y
    y = y.to(s["c"].dtype)
    return y, torch.maximum(s["amax"], y.abs().amax().float())


def _seen(codes, scales, fmt):
    """Codes and scales as the values they stand for (views, no copies)."""
    return codes.view(F8[fmt]), scales.view(torch.float8_e8m0fnu) if scales.dtype == torch.uint8 else scales


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "quantize":
        out = {}
        if s["row"]:
            out["row"] = _seen(*_quantized(s["x"], s["fmt"], s["pow2"], s["tile"]), s["fmt"])
        if s["col"]:
            out["col"] = _seen(*_quantized(s["x"].t(), s["fmt"], s["pow2"], s["tile"]), s["fmt"])
        return out
    if s["op"] == "product":
        a = _operand_values(s["a"], s["fmt"], False)
        b = _operand_values(s["b"], "e4m3", s["tile"])
        return torch.mm(a, b.t()).to(s["c"].dtype)
    return _plain_dropout(s)


def _run_own(s):
    import fp4_block_scaled_amax_amd as lib

    fmts = {"e4m3": lib.E4M3, "e5m2": lib.E5M2}
    if s["op"] == "quantize":
        f = fmts[s["fmt"]]
        row = lib.Fp8Quantized(*s["row_out"], cols=s["cols"], fmt=f, tile=s["tile"]) if s["row"] else None
        col = lib.Fp8Quantized(*s["col_out"], cols=s["rows"], fmt=f, tile=s["tile"]) if s["col"] else None
        lib.quantize_fp8(s["x"], row=row, col=col)
        return {n: _seen(*s[n + "_out"], s["fmt"]) for n in ("row", "col") if s[n]}
    if s["op"] == "product":
        a = lib.Fp8Quantized(*s["a"], cols=s["K"], fmt=fmts[s["fmt"]], tile=False)
        b = lib.Fp8Quantized(*s["b"], cols=s["K"], fmt=lib.E4M3, tile=s["tile"])
        return {"fprop": lib.gemm_fp8_fprop, "dgrad": lib.gemm_fp8_dgrad, "wgrad": lib.gemm_fp8_wgrad}[s["role"]](a, b, s["c"])
    if s["backward"]:
        lib.dropout_backward(s["in"], s["p"], s["key"], s["step"], s["c"], amax=s["amax"])
    else:
        lib.dropout(s["in"], s["p"], s["key"], s["step"], s["c"], residual=s["res"], amax=s["amax"])
    return s["c"], s["amax"]


# -------------------------------------------------------------------- work --

def _operand_bytes(rows, cols, pow2, tile):
    blocks = (cols + 127) // 128 * ((rows + 127) // 128 if tile else rows)
    return rows * cols + blocks * (1 if pow2 else 4)


def work(case):
    if case["op"] == "quantize":
        R, C = case["rows"], case["cols"]
        b = 2 * R * C
        b += _operand_bytes(R, C, case["pow2"], case["tile"]) if case["row"] else 0
        b += _operand_bytes(C, R, case["pow2"], case["tile"]) if case["col"] else 0
        return {"bytes": b, "flops": 4 * R * C}
    if case["op"] == "product":
        M, N, K = _mnk(case)
        return {"bytes": _operand_bytes(M, K, case["pow2"], False) + _operand_bytes(N, K, case["pow2"], case["tile"])
                + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    n, size = case["rows"] * case["cols"], {"bf16": 2, "f32": 4}
    return {"bytes": n * (size[case["x"]] + size[case["out"]] * (2 if case["residual"] else 1)), "flops": 3 * n}


# ----------------------------------------------------- the definition, fp64 --

def _exact_operand(x, case):
    """Codes' values and scales of x blocked along its columns: the nearest values of the format to x / s."""
    fmt, f = case["fmt"], LARGEST[case["fmt"]]
    bits, least = (3, -6) if fmt == "e4m3" else (2, -14)
    R, C = x.shape
    x = torch.nn.functional.pad(x.double(), (0, up(C) - C))
    a = x.abs().reshape(R, -1, 128).amax(2)                                  # [R][blocks]
    if case["tile"]:
        a = torch.nn.functional.pad(a, (0, 0, 0, up(R) - R)).reshape(-1, 128, a.shape[1]).amax(1)
    s = a / f
    s = torch.exp2(torch.ceil(torch.log2(s.clamp(min=2.0 ** -127)))) if case["pow2"] else s.clamp(min=2.0 ** -126)
    each = s.repeat_interleave(128, 0)[:R] if case["tile"] else s
    v = x / each.repeat_interleave(128, 1)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** least))) - bits)
    return torch.round(v / step).mul(step).clamp(-f, f), s.t().contiguous()


def _exact_product_operand(q, fmt, tile):
    codes, scales = q
    s = scales.double() if scales.dtype != torch.uint8 else torch.exp2(scales.double() - 127)
    at = torch.arange(codes.shape[0], device="cuda") // (128 if tile else 1)
    block = torch.arange(codes.shape[1], device="cuda") // 128
    return codes.view(F8[fmt]).double() * s[block][:, at].t()


def _exact_keep(n, key, offset, t):
    """Philox4x32-10 with the 32 x 32-bit products from 16-bit limbs, two products side by side."""
    calls = torch.arange((n + 7) // 8, dtype=torch.int64, device="cuda")
    even = torch.stack([calls % 2 ** 32, torch.full_like(calls, offset)])     # words 0 and 2
    odd = torch.stack([calls // 2 ** 32, torch.full_like(calls, 2)])          # words 1 and 3
    mul = torch.tensor([[0xD2511F53], [0xCD9E8D57]], dtype=torch.int64, device="cuda")
    key = torch.tensor([[key % 2 ** 32], [key // 2 ** 32 % 2 ** 32]], dtype=torch.int64, device="cuda")
    bump = torch.tensor([[0x9E3779B9], [0xBB67AE85]], dtype=torch.int64, device="cuda")
    for _ in range(10):
        low, high = mul * (even % 65536), mul * (even // 65536)               # below 2^48 each
        mid = high + low // 65536
        lo, hi = (mid % 65536) * 65536 + low % 65536, mid // 65536
        even, odd = hi.flip(0) ^ odd ^ key, lo.flip(0)
        key = (key + bump) % 2 ** 32
    words = torch.stack([even[0], odd[0], even[1], odd[1]], 1)
    return torch.stack([words % 65536, words // 65536], 2).flatten()[:n] >= t


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return {n: _exact_operand(x, case) for n, x in (("row", s["x"]), ("col", s["x"].t())) if case[n]}
    if case["op"] == "product":
        return torch.mm(_exact_product_operand(s["a"], case["fmt"], False),
                        _exact_product_operand(s["b"], "e4m3", case["tile"]).t().contiguous())
    t = round(65536 * case["p"])
    keep = _exact_keep(s["in"].numel(), s["key"], s["step"], t).view(s["in"].shape)
    y = torch.where(keep, s["in"].double() * 65536 / (65536 - t), 0.0)
    # the amax is that of the stored, rounded values: it has no value of its own in 64 bits
    return (y if s["res"] is None else y + s["res"].double()), None
