"""The linears of routed experts on FP4 operands, and products of unquantized tokens with FP4 weights: cases, plain forms and calls.

Operators (rows of tokens sorted by expert; expert g owns rows offsets[g] .. offsets[g + 1] - 1):
  * quantize: bf16 rows, gathered by an index or in place, to E2M1 codes with one UE5M3 scale per block of 16 under a
    tensor scale, as the row-wise operand (blocked along the columns) and / or the transposed operand (blocked along
    each expert's rows); the answer is the operands' values and the running amax;
  * product: fprop, dgrad and wgrad of the experts' linears on such operands;
  * tokens: bf16 tokens times FP4 weights, of one linear or of the experts that the tokens are routed to.

Layouts.  An R x C operand: codes [R][C / 2] (element 2j in the low nibble), scales [R][C / 16], values ts * s * q.
The transposed operand of T grouped rows has 128 * (ceil(T / 128) + experts) columns: expert g's rows begin at column
128 * (ceil(offsets[g] / 128) + g), zeros follow up to the next multiple of 128, and no other column is read or written.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def up(n, k=128):
    return (n + k - 1) // k * k


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # 8192 tokens, two experts each, gathered into the up projection's input; both operands from one read
        dict(name="quantize routed activations", op="quantize", rows=16384, tokens=8192, cols=4096, experts=16, skew=0.5,
             sr=False, row=True, col=True),
        # the gradient of the experts' hidden layer, stochastically rounded
        dict(name="quantize gradient", op="quantize", rows=16384, tokens=0, cols=2048, experts=16, skew=0.5, sr=True,
             row=True, col=True),
        # a short ragged batch before fprop: latency
        dict(name="quantize few rows", op="quantize", rows=24, tokens=13, cols=4112, experts=8, skew=1.0, sr=False,
             row=True, col=False),
        # up projection of 16 experts, forward
        dict(name="fprop up", op="product", role="fprop", rows=16384, inputs=4096, outputs=2048, experts=16, skew=0.5,
             out="bf16"),
        # a few wide experts, forward
        dict(name="fprop wide", op="product", role="fprop", rows=16384, inputs=4096, outputs=16384, experts=8, skew=0.3,
             out="bf16"),
        # many small experts, input gradient
        dict(name="dgrad many experts", op="product", role="dgrad", rows=16384, inputs=4096, outputs=2048, experts=64,
             skew=0.7, out="f32"),
        # weight gradients of 16 experts
        dict(name="wgrad up", op="product", role="wgrad", rows=16384, inputs=4096, outputs=2048, experts=16, skew=0.5,
             out="f32"),
        # a ragged micro-batch through layers of odd sizes, some experts without a row
        dict(name="fprop ragged", op="product", role="fprop", rows=1531, inputs=2064, outputs=1305, experts=7, skew=2.0,
             out="f32"),
        # one token through a dense up projection (evaluation by generation)
        dict(name="one token", op="tokens", rows=1, inputs=4096, outputs=16384, experts=0, skew=0.0, out="bf16"),
        # sixteen requests at once through a dense down projection
        dict(name="sixteen tokens", op="tokens", rows=16, inputs=16384, outputs=4096, experts=0, skew=0.0, out="bf16"),
        # one token through its 8 of 64 experts
        dict(name="one token, experts", op="tokens", rows=8, inputs=4096, outputs=2048, experts=64, skew=0.0, out="bf16"),
        # a small batch through layers of odd sizes
        dict(name="batch, odd experts", op="tokens", rows=61, inputs=2064, outputs=1305, experts=9, skew=1.0, out="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "tokens", "tokens"])
    experts, skew = _log(rng, 1, 64), round(rng.uniform(0.0, 2.0), 2)
    if op == "quantize":
        rows = _log(rng, 1, 16384)
        outputs = rng.choice(["row", "col", "both", "both"])
        return dict(op=op, rows=rows, tokens=rng.choice([0, max(1, rows // 2)]), cols=16 * _log(rng, 1, 256), experts=experts,
                    skew=skew, sr=rng.random() < 0.5, row=outputs != "col", col=outputs != "row")
    if op == "product":
        role = rng.choice(["fprop", "dgrad", "wgrad"])
        inputs = _log(rng, 128, 8192) if role == "wgrad" else 16 * _log(rng, 8, 512)
        outputs = 16 * _log(rng, 8, 512) if role == "dgrad" else _log(rng, 128, 8192)
        experts = min(experts, max(1, 64 * 4096 * 2048 // (inputs * outputs)))
        return dict(op=op, role=role, rows=_log(rng, 1, 16384), inputs=inputs, outputs=outputs, experts=experts, skew=skew,
                    out=rng.choice(["bf16", "f32"]))
    inputs, outputs = 16 * _log(rng, 8, 1024), _log(rng, 64, 16384)
    experts = min(experts, 64 * 4096 * 2048 // (inputs * outputs)) if rng.random() < 0.6 else 0
    return dict(op=op, rows=_log(rng, 1, 64), inputs=inputs, outputs=outputs, experts=experts, skew=skew,
                out=rng.choice(["bf16", "f32"]))


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


def _counts(rows, experts, skew, gen):
    """Rows of each expert: every row draws its expert, with unequal odds."""
    odds = torch.softmax(skew * torch.randn(experts, generator=gen, device="cuda"), 0)
    to = torch.multinomial(odds, rows, replacement=True, generator=gen)
    return torch.bincount(to, minlength=experts).tolist()


def _tensor_scale(x):
    """The tensor scale that a refresh from x's own amax leaves: amax / (6 * 7168)."""
    return x.abs().amax().float().reshape(1) / torch.full((1,), 6.0 * 7168.0, device=x.device)


def _placed(counts):
    """(columns of the transposed operand, the column of each grouped row)."""
    first, at = 0, []
    for g, n in enumerate(counts):
        p = up(first) + 128 * g
        at.append(torch.arange(p, p + n))
        first += n
    return up(first) + 128 * len(counts), torch.cat(at).cuda()


def _packed(x, ts):
    """(codes, scales) of x's rows, quantized to nearest."""
    q, s = _quantized(x.float(), ts, None)
    e = (q.abs() * 2).to(torch.int64)                     # 0 1 2 3 4 6 8 12
    e = torch.tensor([0, 1, 2, 3, 4, 4, 5, 5, 6, 6, 6, 6, 7], device=x.device)[e] + 8 * torch.signbit(q)
    return (e[:, 0::2] + 16 * e[:, 1::2]).to(torch.uint8), s.to(torch.uint8)


def _packed_in_slices(make, n, ts):
    got = [_packed(make(i), ts[i:i + 1] if ts.numel() > 1 else ts) for i in range(n)]
    return tuple(torch.stack(v) for v in zip(*got))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case, seed=seed)
    T, E = case["rows"], case["experts"]
    if E:
        s["counts"] = _counts(T, E, case["skew"], gen)
        ends = torch.cumsum(torch.tensor([0] + s["counts"]), 0)
        s["offsets"] = ends.to(torch.int32).cuda()
        s["ends"] = ends.tolist()
    if case["op"] == "quantize":
        C, X = case["cols"], case["tokens"] or T
        s["x"] = _values("gradient" if case["sr"] else "activation", X, C, gen)
        s["index"] = torch.randint(0, X, (T,), generator=gen, device="cuda").to(torch.int32) if case["tokens"] else None
        s["ts"], s["amax"] = _tensor_scale(s["x"]), torch.zeros(1, device="cuda")
        P, s["at"] = _placed(s["counts"])
        s["shapes"] = {n: v for n, v in (("row", (T, C)), ("col", (C, P))) if case[n]}
        s["buffers"] = {n: (torch.zeros((r, c // 2), dtype=torch.uint8, device="cuda"),
                            torch.zeros((r, c // 16), dtype=torch.uint8, device="cuda"),
                            torch.empty((r, c), device="cuda")) for n, (r, c) in s["shapes"].items()}
        s["key"], s["step"] = 0x9E3779B97F4A7C15 ^ (seed * 0x2545F491), 7 + seed % 1000
        return s
    i, o, n = case["inputs"], case["outputs"], max(1, E)
    out = TYPES[case["out"]]
    if case["op"] == "product" and case["role"] == "wgrad":
        P, at = _placed(s["counts"])
        for name, kind, width in (("a", "gradient", o), ("b", "activation", i)):
            x = _values(kind, T, width, gen)
            wide = torch.zeros((width, P), dtype=x.dtype, device="cuda").index_copy_(1, at, x.t())
            s[name + "_ts"] = _tensor_scale(x)
            s[name] = _packed(wide, s[name + "_ts"])
        s["c"] = torch.empty((n, o, i), dtype=out, device="cuda")
        return s
    N, K = (i, o) if case["op"] == "product" and case["role"] == "dgrad" else (o, i)
    s["K"], s["N"] = K, N
    s["b_ts"] = 0.02 * 6.0 / (6.0 * 7168.0) * torch.exp(0.1 * torch.randn(n, generator=gen, device="cuda"))
    s["b"] = _packed_in_slices(lambda g: _values("weight", N, K, gen), n, s["b_ts"])
    x = _values("gradient" if case.get("role") == "dgrad" else "activation", T, K, gen)
    if case["op"] == "product":
        s["a_ts"] = _tensor_scale(x)
        s["a"] = _packed(x, s["a_ts"])
        s["amax"] = torch.zeros(1, device="cuda") if case["out"] == "bf16" else None
    else:
        s["x"] = x
    s["c"] = torch.empty((T, N), dtype=out, device="cuda")
    return s


# -------------------------------------------------------------- plain forms --

MASK = 0xFFFFFFFF


def _round(c, k):
    """One Philox round; the products wrap in 64 bits, their halves are masked out."""
    p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
    return [((p1 >> 32) & MASK) ^ c[1] ^ k[0], p1 & MASK, ((p0 >> 32) & MASK) ^ c[3] ^ k[1], p0 & MASK]


def _random16(shape, key, offset, orientation):
    """The 16 random bits of each element of an output of this shape."""
    call = torch.arange((shape[0] * shape[1] + 7) // 8, dtype=torch.int64, device="cuda")
    c = [call & MASK, call >> 32, torch.full_like(call, offset), torch.full_like(call, orientation)]
    k0, k1 = key & MASK, (key >> 32) & MASK
    for r in range(10):
        c = _round(c, ((k0 + r * 0x9E3779B9) & MASK, (k1 + r * 0xBB67AE85) & MASK))
    return torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], dim=1).view(-1)[:shape[0] * shape[1]].view(shape)


def _scale_values(codes):
    """UE5M3 bytes (as integers) to values."""
    c = codes.to(torch.int32)                             # a byte is the top of an fp32 number with another bias
    return torch.where(c < 8, c.float() * 2.0 ** -17, ((c << 20) + (112 << 23)).view(torch.float32))


def _quantized(x, ts, u):
    """(payload values, scale codes) of the blocks of 16 along x's rows: nearest, or by the 16 random bits u."""
    R, C = x.shape
    b = x.view(R, C // 16, 16)
    s = b.abs().amax(2) / (6.0 * ts)
    bits = s.view(torch.int32)
    normal = (((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - 896).clamp(max=254)
    code = torch.where(s < 2.0 ** -14, torch.round(s * 2.0 ** 17).clamp(max=8).to(torch.int32), normal)
    r = torch.where(code == 0, torch.zeros_like(s), 1.0 / (ts * _scale_values(code)))
    v = (b * r.unsqueeze(2)).view(R, C)
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    if u is None:
        q = torch.round(a / step) * step                  # to even steps, which are the grid's even codes
    else:
        low = torch.floor(a / step) * step
        q = torch.where(u.float() < 65536.0 * ((a - low) / step), low + step, low)
    return torch.copysign(q, x), code


def _plain_quantize(s):
    x = s["x"].float()
    x = x if s["index"] is None else x[s["index"].long()]
    out = {"amax": torch.maximum(s["amax"], x.abs().amax())}
    for n, orientation in (("row", 0), ("col", 1)):
        if not s[n]:
            continue
        y = x if n == "row" else torch.zeros(s["shapes"]["col"], device="cuda").index_copy_(1, s["at"], x.t())
        u = _random16(s["shapes"][n], s["key"], s["step"], orientation) if s["sr"] else None
        q, code = _quantized(y, s["ts"], u)
        out[n] = (q.view(*code.shape, 16) * _scale_values(code).unsqueeze(2)).view(q.shape) * s["ts"]
    return out


def _unpacked(codes, scales):
    """q * s of an operand."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    pairs = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], 1)          # of each byte
    q = pairs[codes.long()].view(*scales.shape, 16)
    return (q * _scale_values(scales).unsqueeze(-1)).view(*codes.shape[:-1], -1)


def _plain_wgrad(s):
    a, b = _unpacked(*s["a"]) * s["a_ts"], _unpacked(*s["b"]) * s["b_ts"]
    c = torch.empty(s["c"].shape, device="cuda")
    for g, n in enumerate(s["counts"]):
        p = up(s["ends"][g]) + 128 * g
        torch.mm(a[:, p:p + n], b[:, p:p + n].t(), out=c[g])
    return c.to(s["c"].dtype)


def _plain_rows(s, x):
    """x's rows times the weights of the expert that owns them."""
    if not s["experts"]:
        return torch.mm(x, (_unpacked(s["b"][0][0], s["b"][1][0]) * s["b_ts"]).t()).to(s["c"].dtype)
    c = torch.empty(s["c"].shape, device="cuda")
    for g, n in enumerate(s["counts"]):
        if n:
            w = _unpacked(s["b"][0][g], s["b"][1][g]) * s["b_ts"][g]
            torch.mm(x[s["ends"][g]:s["ends"][g] + n], w.t(), out=c[s["ends"][g]:s["ends"][g] + n])
    return c.to(s["c"].dtype)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "quantize":
        return _plain_quantize(s)
    if s["op"] == "tokens":
        return _plain_rows(s, s["x"].float())
    if s["role"] == "wgrad":
        return _plain_wgrad(s)
    c = _plain_rows(s, _unpacked(*s["a"]) * s["a_ts"])
    return (c, torch.maximum(s["amax"], c.abs().amax().float())) if s["amax"] is not None else c


def _run_own(s):
    import fp4_block_scaled_amax_amd as lib

    if s["op"] == "quantize":
        q = {n: lib.Quantized(b[0], b[1], s["ts"]) for n, b in s["buffers"].items()}
        lib.quantize_grouped(s["x"], s["offsets"], s["ts"], lib.SR if s["sr"] else lib.RNE, s["key"], s["step"],
                             row=q.get("row"), col=q.get("col"), index=s["index"], amax=s["amax"])
        return {"amax": s["amax"], **{n: lib.dequantize(v, s["buffers"][n][2]) for n, v in q.items()}}
    if s["op"] == "tokens":
        if not s["experts"]:
            return lib.gemm_weight_only(s["x"], lib.Quantized(s["b"][0][0], s["b"][1][0], s["b_ts"]), s["c"])
        return lib.gemm_weight_only(s["x"], lib.ExpertWeights(*s["b"], s["b_ts"]), s["c"], offsets=s["offsets"])
    a = lib.Quantized(*s["a"], s["a_ts"])
    if s["role"] == "wgrad":
        return lib.gemm_grouped_wgrad(a, lib.Quantized(*s["b"], s["b_ts"]), s["offsets"], s["c"])
    w = lib.ExpertWeights(*s["b"], s["b_ts"])
    call = lib.gemm_grouped_fprop if s["role"] == "fprop" else lib.gemm_grouped_dgrad
    call(a, w, s["offsets"], s["c"], amax=s["amax"])
    return (s["c"], s["amax"]) if s["amax"] is not None else s["c"]


# -------------------------------------------------------------------- work --

def work(case):
    T, E, size = case["rows"], case["experts"], {"bf16": 2, "f32": 4}
    if case["op"] == "quantize":
        C, P = case["cols"], up(T) + 128 * E
        b = 2 * min(case["tokens"] or T, T) * C + (4 * T * C if case["row"] else 0) + (4 * C * P if case["col"] else 0)
        return {"bytes": b, "flops": 4 * T * C}
    i, o = case["inputs"], case["outputs"]
    held = min(max(1, E), T)                              # experts whose weights are read, at most
    if case["op"] == "tokens":
        return {"bytes": 2 * T * i + 9 * held * i * o // 16 + size[case["out"]] * T * o, "flops": 2 * T * i * o}
    if case["role"] == "wgrad":
        return {"bytes": 9 * T * (i + o) // 16 + size[case["out"]] * E * i * o, "flops": 2 * T * i * o}
    K, N = (i, o) if case["role"] == "fprop" else (o, i)
    return {"bytes": 9 * (T * K + held * N * K) // 16 + size[case["out"]] * T * N, "flops": 2 * T * N * K}


# ----------------------------------------------------- the definition, fp64 --

def _exact_scale(s):
    """The nearest UE5M3 value to s (ties to the even mantissa), saturating."""
    step = torch.exp2(torch.floor(torch.log2(s.clamp(min=2.0 ** -14))) - 3)
    return (torch.round(s / step) * step).clamp(max=114688.0)


def _exact_bits(n, key, offset, orientation):
    """Philox4x32-10 with the 32 x 32-bit products from 16-bit limbs, two products side by side."""
    calls = torch.arange((n + 7) // 8, dtype=torch.int64, device="cuda")
    even = torch.stack([calls % 2 ** 32, torch.full_like(calls, offset)])          # words 0 and 2
    odd = torch.stack([calls // 2 ** 32, torch.full_like(calls, orientation)])     # words 1 and 3
    mul = torch.tensor([[0xD2511F53], [0xCD9E8D57]], dtype=torch.int64, device="cuda")
    key = torch.tensor([[key % 2 ** 32], [key // 2 ** 32 % 2 ** 32]], dtype=torch.int64, device="cuda")
    bump = torch.tensor([[0x9E3779B9], [0xBB67AE85]], dtype=torch.int64, device="cuda")
    for _ in range(10):
        low, high = mul * (even % 65536), mul * (even // 65536)                    # below 2^48 each
        mid = high + low // 65536
        lo, hi = (mid % 65536) * 65536 + low % 65536, mid // 65536
        even, odd = hi.flip(0) ^ odd ^ key, lo.flip(0)
        key = (key + bump) % 2 ** 32
    words = torch.stack([even[0], odd[0], even[1], odd[1]], 1)
    return torch.stack([words % 65536, words // 65536], 2).flatten()[:n]


def _stored(v):
    """The 32-bit value that the definition names at this step: one rounding of the 64-bit one."""
    return v.float().double()


def _exact_values(x, ts, u):
    """ts * s * q of the blocks of 16 along x's rows.  The codes hang on the definition's intermediate values (amax / (6
    ts), 1 / (ts * s) and their product with x, which meets the payload grid's borders), so these are rounded as it says."""
    b = x.view(x.shape[0], -1, 16)
    s = _exact_scale(_stored(b.abs().amax(2) / _stored(6.0 * ts))).unsqueeze(2)
    a = torch.where(s == 0, 0.0, _stored(b.abs() * _stored(1.0 / _stored(ts * s)))).clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=1.0, max=4.0))) - 1)
    if u is None:
        q = torch.round(a / step) * step
    else:
        low = torch.floor(a / step)
        q = (low + (u.view(b.shape) < 65536 * (a / step - low))) * step
    return (torch.sign(b) * q * s * ts).view(x.shape)


def _exact_operand(codes, scales):
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).to(torch.int64)
    m, e = (c % 2).double(), (c // 2 % 4).double()
    q = torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2)) * (1 - 2 * (c // 8).double())
    f, e = (scales % 8).double(), (scales // 8).double()
    s = torch.where(e == 0, f * 2.0 ** -17, torch.exp2(e - 15) * (1 + f / 8))
    return (q.view(*s.shape, 16) * s.unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x, ts = s["x"].double(), s["ts"].double()
        x = x if s["index"] is None else x.index_select(0, s["index"].long())
        out = {"amax": x.abs().max().reshape(1)}
        if case["row"]:
            u = _exact_bits(x.numel(), s["key"], s["step"], 0) if case["sr"] else None
            out["row"] = _exact_values(x, ts, u)
        if case["col"]:
            C, P = s["shapes"]["col"]
            y = torch.zeros((P, C), dtype=torch.float64, device="cuda")
            y[s["at"]] = x
            u = _exact_bits(C * P, s["key"], s["step"], 1) if case["sr"] else None
            out["col"] = _exact_values(y.t().contiguous(), ts, u)
        return out
    if case["op"] == "product" and case["role"] == "wgrad":
        a, b = _exact_operand(*s["a"]), _exact_operand(*s["b"])
        spans = [(up(s["ends"][g]) + 128 * g, n) for g, n in enumerate(s["counts"])]
        return torch.stack([torch.mm(a[:, p:p + n], b[:, p:p + n].t().contiguous()) for p, n in spans]) * (s["a_ts"].double() * s["b_ts"].double())
    x = s["x"].double() if case["op"] == "tokens" else _exact_operand(*s["a"]) * s["a_ts"].double()
    spans = list(zip(s["ends"], s["counts"])) if case["experts"] else [(0, case["rows"])]
    c = torch.cat([torch.mm(x[p:p + n], _exact_operand(s["b"][0][g], s["b"][1][g]).t().contiguous()) * s["b_ts"][g].double()
                   for g, (p, n) in enumerate(spans)])
    # the amax is that of the stored, rounded values: it has no value of its own in 64 bits
    return (c, None) if case["op"] == "product" and s["amax"] is not None else c
