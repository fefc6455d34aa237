"""The 8-bit and 4-bit floating point operators around the quantized linear layer, as cases to measure.

Three operators, each in its plain form (elementary torch operations) and as the library's calls:

* "norm": the residual's addition and the root-mean-square norm in front of a quantized projection,
  with the normed row written in bf16/fp32 and quantized: int8 codes with one scale per token (8 or 6
  bits), or MXFP4 (bits = 4).
* "quantize": MXFP4 of a matrix and back: 4-bit codes (E2M1) with one power-of-two scale (E8M0) for each
  32 consecutive channels of a row.
* "linear": Y = MXFP4(X * s_inv) . Wᵀ with W held in MXFP4, fp32 sums.

Quantized outputs are returned as the values they stand for, in bf16.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
_DTYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # one decoded token through the input norm of the 2B layer set
        dict(name="norm8 decode 1x1536", op="norm", T=1, d=1536, bits=8, dtype="bf16", residual=True, smooth=True),
        # a prompt in fp32 without a residual, of a width that is no power of two
        dict(name="norm8 f32 300x8960", op="norm", T=300, d=8960, bits=8, dtype="f32", residual=False, smooth=True),
        # the 72B layer set's prompt, A6
        dict(name="norm6 prompt 8192x8192", op="norm", T=8192, d=8192, bits=6, dtype="bf16", residual=True, smooth=True),
        # a decode batch, the row leaving in MXFP4
        dict(name="norm4 decode 16x8192", op="norm", T=16, d=8192, bits=4, dtype="bf16", residual=True, smooth=False),
        # the 2B layer set's prompt, MXFP4
        dict(name="norm4 prompt 2048x1536", op="norm", T=2048, d=1536, bits=4, dtype="bf16", residual=True, smooth=True),
        # the 2B down projection's activations, an odd number of rows
        dict(name="quantize act 2047x8960", op="quantize", rows=2047, cols=8960, dtype="bf16", smooth=True),
        # weights of the 72B gate projection, once for each model
        dict(name="quantize weight 29568x8192", op="quantize", rows=29568, cols=8192, dtype="bf16", smooth=True),
        # one decoded token of the 72B key projection
        dict(name="linear decode 1x8192x1024", op="linear", T=1, K=8192, N=1024, x="bf16", y="bf16", smooth=True),
        # a decode batch through the 72B down projection
        dict(name="linear decode 16x29568x8192", op="linear", T=16, K=29568, N=8192, x="bf16", y="bf16", smooth=True),
        # a short prompt through the 8B qkv projection, fp32 in and out
        dict(name="linear f32 130x4096x6144", op="linear", T=130, K=4096, N=6144, x="f32", y="f32", smooth=False),
        # the 2B gate projection at the 2B set's prompt
        dict(name="linear 2048x1536x8960", op="linear", T=2048, K=1536, N=8960, x="bf16", y="bf16", smooth=True),
        # the 72B gate projection at the 72B set's prompt
        dict(name="linear 8192x8192x29568", op="linear", T=8192, K=8192, N=29568, x="bf16", y="bf16", smooth=True),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        bits = rng.choice([8, 6, 4])
        d = 32 * _between(rng, 4, 512)
        if bits != 4:
            d += 8 * rng.randrange(4)
        return dict(op=op, T=_between(rng, 1, 8192 if d <= 8192 and dtype == "bf16" else 3500), d=d, bits=bits, dtype=dtype,
                    residual=rng.random() < 0.7, smooth=rng.random() < 0.5)
    if op == "quantize":
        cols = 32 * _between(rng, 1, 924)
        rows = _between(rng, 1, min(29568, 29568 * 8192 // cols // (1 if dtype == "bf16" else 2)))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, smooth=rng.random() < 0.5)
    T = _between(rng, 1, 8192)
    K = 32 * _between(rng, 2, 924)
    N = _between(rng, 64, min(29568, 8192 * 8192 * 29568 // (T * K)))
    return dict(op=op, T=T, K=K, N=N, x=dtype, y=rng.choice(["bf16", "bf16", "f32"]), smooth=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).mul_(std)


def _activations(T, d, g):
    """N(0, 1) rows with the outliers of a language model's activations: a few channels that are large for every
    token (x20), and a few more, others for each token (x30)."""
    x = _normal((T, d), g)
    always = torch.randperm(d, generator=g, device="cuda")[: max(1, d // 64)]
    x[:, always] *= 20.0
    some = torch.randint(0, d, (T, max(1, d // 128)), generator=g, device="cuda")
    x.scatter_(1, some, x.gather(1, some) * 30.0)
    return x


def _pow2(e):
    """fp32 2^e for whole e in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 0x00400000)).to(torch.int32).view(F32)


def _mx4(v):
    """MXFP4 of fp32 v [rows, cols]: codes [rows, cols] in 0..15 (sign, then E2M1) and the scale exponents
    [rows, cols/32]. The largest magnitude of a block decides: E = floor(log2 max) - 2, in [-127, 127];
    ties of a code go to the even one, and magnitudes beyond 6 * 2^E to 6."""
    rows, cols = v.shape
    b = v.view(rows, cols // 32, 32)
    top = b.abs().amax(-1)
    _, e = torch.frexp(top)  # top = m * 2^e, m in [0.5, 1)
    e = torch.where(top > 0, (e.to(torch.int32) - 3).clamp(-127, 127), torch.full_like(e, -127, dtype=torch.int32))
    a = b.abs() * _pow2(-e).unsqueeze(-1)
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(b).to(torch.uint8) << 3
    return code.view(rows, cols), e


_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(code, e, dtype=F32):
    """The values that codes and scale exponents stand for."""
    rows, cols = code.shape
    table = torch.tensor([*_MAGNITUDES, *(-m for m in _MAGNITUDES)], dtype=F32, device=code.device)
    v = table[code.int()].view(rows, cols // 32, 32) * _pow2(e).unsqueeze(-1)
    return v.view(rows, cols).to(dtype)


def _scale_tiles(e):
    """Scale exponents [rows, blocks] as the bytes that the product reads: tiles of 128 rows x 4 blocks of 512
    bytes, row-major over the matrix, byte (row % 32) * 16 + (row % 128) // 32 * 4 + block % 4 in its tile; rows and
    blocks past the end hold 127 (a scale of one)."""
    rows, blocks = e.shape
    R, B = -(-rows // 128), -(-blocks // 4)
    full = torch.full((R * 128, B * 4), 127, dtype=torch.uint8, device=e.device)
    full[:rows, :blocks] = (e + 127).to(torch.uint8)
    return full.view(R, 4, 32, B, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _scale_rows(tiles, rows, blocks):
    """The scale exponents [rows, blocks] of such bytes."""
    R, B = -(-rows // 128), -(-blocks // 4)
    return tiles.view(R, B, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, B * 4)[:rows, :blocks].to(torch.int32) - 127


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "norm":
        T, d, t = case["T"], case["d"], _DTYPES[case["dtype"]]
        s["x"] = _normal((T, d), g, 0.5).to(t)
        s["r"] = _activations(T, d, g).to(t) if case["residual"] else None
        if not case["residual"]:
            s["x"] = _activations(T, d, g).to(t)
        s["gamma"] = (1.0 + _normal((d,), g, 0.2)).to(t)
        s["s_inv"] = torch.exp(_normal((d,), g, 0.5)) if case["smooth"] else None
        s["eps"] = 1e-6
    elif case["op"] == "quantize":
        s["v"] = _activations(case["rows"], case["cols"], g).to(_DTYPES[case["dtype"]])
        s["s"] = torch.exp(_normal((case["cols"],), g, 0.5)) if case["smooth"] else None
    else:
        T, K, N = case["T"], case["K"], case["N"]
        s["v"] = _activations(T, K, g).to(_DTYPES[case["x"]])
        s["s_inv"] = torch.exp(_normal((K,), g, 0.5)) if case["smooth"] else None
        code, e = _mx4(_normal((N, K), g, 0.02))
        s["w_codes"] = code[:, 0::2] | code[:, 1::2] << 4  # two codes in a byte, the even channel low
        s["w_scales"] = _scale_tiles(e)
    return s


# ---------------------------------------------------------------- one pass

def _norm_plain(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    # the statistic in 64 bits, rounded once: every value next to a border of a code hangs on it
    rstd = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + s["eps"])).float()
    y = (h * rstd) * s["gamma"].float()
    v = y if s["s_inv"] is None else y * s["s_inv"]
    out = {"y": y.to(s["x"].dtype)}
    if s["r"] is not None:
        out["residual"] = h.to(s["x"].dtype)
    if s["bits"] == 4:
        out["values"] = _values(*_mx4(v), BF16)
    else:
        qmax = float(2 ** (s["bits"] - 1) - 1)
        sa = v.abs().amax(-1, keepdim=True) / qmax
        q = torch.where(sa > 0, torch.round(v / sa).clamp(-qmax, qmax), torch.zeros_like(v))
        out["values"] = (q * sa).to(BF16)
        out["sa"] = sa.view(-1)
    return out


def _norm_own(s):
    import quantized_gemm_moe_b200 as qe
    x, (T, d) = s["x"], s["x"].shape
    y = torch.empty_like(x)
    h = torch.empty_like(x) if s["r"] is not None else None
    values = torch.empty((T, d), dtype=BF16, device=x.device)
    out = {"y": y, "values": values}
    if s["bits"] == 4:
        codes = torch.empty((T, d // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty(qe.mx4_scale_bytes(T, d), dtype=torch.uint8, device=x.device)
    else:
        codes = torch.empty((T, d), dtype=torch.int8, device=x.device)
        scales = out["sa"] = torch.empty(T, dtype=F32, device=x.device)
    qe.add_rmsnorm_quant(x, s["gamma"], s["eps"], s["bits"], codes, scales, residual=s["r"], residual_out=h, Y=y, s_inv=s["s_inv"])
    if s["bits"] == 4:
        qe.mx4_dequantize(codes, scales, values)
    else:
        qe.act_dequant(codes, scales, values)
    if h is not None:
        out["residual"] = h
    return out


def _quantize_plain(s):
    v = s["v"].float()
    return _values(*_mx4(v if s["s"] is None else v * s["s"]), BF16)


def _quantize_own(s):
    import quantized_gemm_moe_b200 as qe
    v, (rows, cols) = s["v"], s["v"].shape
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=v.device)
    scales = torch.empty(qe.mx4_scale_bytes(rows, cols), dtype=torch.uint8, device=v.device)
    qe.mx4_quantize(v, codes, scales, s=s["s"])
    values = torch.empty((rows, cols), dtype=BF16, device=v.device)
    qe.mx4_dequantize(codes, scales, values)
    return values


def _linear_plain(s):
    v = s["v"].float()
    x = _values(*_mx4(v if s["s_inv"] is None else v * s["s_inv"]))
    c = s["w_codes"]
    code = torch.stack((c & 15, c >> 4), -1).view(s["N"], s["K"])
    w = _values(code, _scale_rows(s["w_scales"], s["N"], s["K"] // 32))
    return (x @ w.T).to(_DTYPES[s["y"]])


def _linear_own(s):
    import quantized_gemm_moe_b200 as qe
    x = s["v"]
    Y = torch.empty((s["T"], s["N"]), dtype=_DTYPES[s["y"]], device=x.device)
    workspace = torch.empty(qe.mx4_linear_workspace_bytes(s["T"], s["K"]), dtype=torch.uint8, device=x.device)
    qe.mx4_linear_forward(s["w_codes"], s["w_scales"], x, Y, workspace, s_inv=s["s_inv"])
    return Y


def run(state):
    if own:
        return {"norm": _norm_own, "quantize": _quantize_own, "linear": _linear_own}[state["op"]](state)
    return {"norm": _norm_plain, "quantize": _quantize_plain, "linear": _linear_plain}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "norm":
        n, b = case["T"] * case["d"], 2 if case["dtype"] == "bf16" else 4
        rows = n * b * (4 if case["residual"] else 2)  # x, y and, with a residual, r and h
        fixed = case["d"] * (b + (4 if case["smooth"] else 0))
        return {"bytes": rows + fixed + 2 * n + (4 * case["T"] if case["bits"] != 4 else 0), "flops": 8 * n}
    if case["op"] == "quantize":
        n, b = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * b + 2 * n + (4 * case["cols"] if case["smooth"] else 0), "flops": 3 * n}
    T, K, N = case["T"], case["K"], case["N"]
    xb, yb = (2 if case[k] == "bf16" else 4 for k in ("x", "y"))
    return {"bytes": T * K * xb + N * K // 2 + N * K // 32 + T * N * yb + (4 * K if case["smooth"] else 0), "flops": 2 * T * K * N}


# ---------------------------------------------------------------- the definition in 64 bits

def _mx4_64(v):
    """The MXFP4 values of v in 64 bits: each block on the grid 0, .5, 1, 1.5, 2, 3, 4, 6 times a power of two."""
    rows, cols = v.shape
    b = v.double().view(rows, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    # the exponent field of a double: floor(log2 top), and -1023 for zero
    power = (top.view(torch.int64) >> 52) - 1023
    unit = ((power - 2).clamp(-127, 127) + 1023 << 52).view(torch.float64)
    a = b.abs() / unit
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return (torch.copysign((torch.round(a / step) * step).clamp_max(6.0), b) * unit).view(rows, cols)


def _once(v):
    """The smoothed value that is quantized is by definition one fp32 product: rounded once."""
    return v.float().double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        v = s["v"].double()
        return _mx4_64(v if s["s"] is None else _once(v * s["s"].double()))
    if case["op"] == "linear":
        x = s["v"].double()
        x = _mx4_64(x if s["s_inv"] is None else _once(x * s["s_inv"].double()))
        N, K = case["N"], case["K"]
        grid = torch.tensor(_MAGNITUDES, dtype=torch.float64, device="cuda")
        w = torch.empty((N, K), dtype=torch.float64, device="cuda")
        for half in (0, 1):
            c = (s["w_codes"] >> (4 * half)) & 15
            w[:, half::2] = grid[(c & 7).int()] * torch.where(c > 7, -1.0, 1.0)
        row, block = torch.arange(N, device="cuda").view(-1, 1), torch.arange(K // 32, device="cuda").view(1, -1)
        at = ((row // 128) * (-(-K // 128)) + block // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + block % 4
        w.view(N, -1, 32).mul_((s["w_scales"][at].long() - 127 + 1023 << 52).view(torch.float64).unsqueeze(-1))
        return x @ w.T
    h = s["x"].double()
    if s["r"] is not None:
        h = h + s["r"].double()
    y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["d"] + s["eps"]) * s["gamma"].double()
    v = y if s["s_inv"] is None else y * s["s_inv"].double()
    out = {"y": y}
    if s["r"] is not None:
        out["residual"] = h
    if case["bits"] == 4:
        out["values"] = _mx4_64(v)
    else:
        most = 2 ** (case["bits"] - 1) - 1
        sa = v.abs().amax(-1) / most
        out["sa"] = sa
        out["values"] = torch.round(v / sa.unsqueeze(-1)).clamp(-most, most) * sa.unsqueeze(-1)
    return out
