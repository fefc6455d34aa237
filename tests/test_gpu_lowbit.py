"""Parity of the norm with quantized output, of MXFP4 and of its product with 64-bit definitions
(oracle/lowbit.py), and their behaviour at the edges: ragged sizes, empty calls, values that are not finite,
streams, captured graphs, memory around the outputs."""
import numpy as np
import pytest
import torch

import oracle
import quantized_gemm_moe_b200 as qe
from oracle import lowbit
from gpu_util import cuda

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rnd(shape, seed, dtype=F32, spread=2.0):
    """Normal values with per-row and per-column factors over a few binades, rounded to dtype; fp32 numpy and cuda."""
    g = np.random.default_rng(seed)
    v = g.standard_normal(shape) * np.exp(g.standard_normal((shape[0], 1)) * spread)
    if len(shape) > 1:
        v = v * np.exp(g.standard_normal((1, shape[1])) * 0.5)
    t = torch.from_numpy(v.astype(np.float32)).to(dtype)
    return t.float().numpy(), t.cuda()


def quantize(X, s=None):
    rows, cols = X.shape
    codes = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((qe.mx4_scale_bytes(rows, cols),), 0xEE, dtype=torch.uint8, device="cuda")
    qe.mx4_quantize(X, codes, scales, s=s)
    return codes, scales


def check_mx4(codes, scales, v):
    """codes and scale tiles equal the definition's for the fp32 values v; bytes of absent rows are untouched."""
    code, scale = lowbit.mx4_quantize(v)
    rows, cols = v.shape
    assert np.array_equal(codes.cpu().numpy(), lowbit.pack_codes(code))
    got = scales.cpu().numpy()
    assert np.array_equal(got[lowbit.scale_offsets(rows, cols)], scale)
    # blocks past the row's end (up to the tile's 128 channels) hold 127
    wide = lowbit.scale_offsets(rows, -(-cols // 128) * 128)
    assert (got[wide[:, cols // 32:]] == 127).all()
    rest = np.ones(got.size, bool)
    rest[wide] = False
    assert (got[rest] == 0xEE).all()
    return code, scale


# ---------------------------------------------------------------- MXFP4

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (128, 128), (129, 160), (33, 1024), (5, 1056), (300, 992), (2, 8960)])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantize_matches_definition(dtype, rows, cols, smooth):
    x, X = rnd((rows, cols), 1 + rows, dtype)
    s = np.exp(np.random.default_rng(2).standard_normal(cols)).astype(np.float32) if smooth else None
    codes, scales = quantize(X, None if s is None else cuda(s))
    v = x if s is None else x * s
    code, scale = check_mx4(codes, scales, v)
    for out in (BF16, F32):  # two significant bits: exact in both
        back = torch.empty((rows, cols), dtype=out, device="cuda")
        qe.mx4_dequantize(codes, scales, back)
        assert np.array_equal(back.double().cpu().numpy(), lowbit.mx4_values(code, scale))


def test_quantize_ties_extremes_and_not_finite():
    x = np.zeros((8, 64), np.float32)
    t = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.99, 4.0], np.float32)
    x[0, :10], x[0, 10:20] = t, -t
    x[1, :10] = np.nextafter(t, np.float32(np.inf))
    x[1, 10:20] = np.nextafter(t, np.float32(0))
    x[2, :10] = t * np.float32(2.0 ** 125)            # the largest scale
    x[3, :10] = t * np.float32(2.0 ** -127)           # the smallest: fp32 subnormals
    x[4, :4] = [1e-45, -1e-45, 3e-39, np.finfo(np.float32).max]
    x[5, 3], x[5, 40] = np.nan, -np.inf
    x[6, :32], x[6, 32:] = np.float32(-0.0), 1.0
    x[7, 0], x[7, 1] = np.finfo(np.float32).max, -1e-30
    codes, scales = quantize(cuda(x))
    code, scale = check_mx4(codes, scales, x)
    back = torch.empty((8, 64), dtype=F32, device="cuda")
    qe.mx4_dequantize(codes, scales, back)
    assert np.array_equal(back.double().cpu().numpy(), lowbit.mx4_values(code, scale), equal_nan=True)
    assert torch.isnan(back[5]).all()


def test_quantize_writes_the_reciprocal_factors():
    x, X = rnd((4, 96), 3)
    s = np.exp(np.random.default_rng(4).standard_normal(96)).astype(np.float32)
    codes, scales = torch.empty((4, 48), dtype=torch.uint8, device="cuda"), torch.empty(512, dtype=torch.uint8, device="cuda")
    s_inv = torch.empty(96, device="cuda")
    qe.mx4_quantize(X, codes, scales, s=cuda(s), s_inv=s_inv)
    assert np.array_equal(s_inv.cpu().numpy(), np.float32(1) / s)


# ---------------------------------------------------------------- norm

def norm_call(X, r, gamma, eps, bits, s_inv, want_y=True, want_h=True):
    T, d = X.shape
    Y = torch.empty_like(X) if want_y else None
    H = torch.empty_like(X) if r is not None and want_h else None
    if bits == 4:
        codes = torch.full((T, d // 2), 0xEE, dtype=torch.uint8, device="cuda")
        scales = torch.full((qe.mx4_scale_bytes(T, d),), 0xEE, dtype=torch.uint8, device="cuda")
    elif bits == 16:
        codes = scales = None
    else:
        codes = torch.empty((T, d), dtype=torch.int8, device="cuda")
        scales = torch.empty(T, device="cuda")
    qe.add_rmsnorm_quant(X, gamma, eps, bits, codes, scales, residual=r, residual_out=H, Y=Y, s_inv=s_inv)
    return H, Y, codes, scales


def rounded(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).double().numpy()


@pytest.mark.parametrize("T,d,bits,xd,gd,res,smooth", [
    (1, 8, 8, BF16, BF16, True, True), (1, 32, 4, BF16, BF16, True, True), (3, 96, 4, F32, F32, False, False),
    (2, 1000, 6, BF16, F32, True, False), (130, 1536, 8, F32, BF16, True, True), (130, 1536, 4, BF16, BF16, False, True),
    (5, 2056, 8, BF16, BF16, True, True), (7, 4096, 16, BF16, BF16, True, False), (7, 4104, 6, F32, F32, True, True),
    (9, 8192, 4, BF16, F32, True, True), (9, 8960, 8, F32, F32, False, True), (3, 16384, 4, F32, BF16, True, False),
    (3, 32768, 8, BF16, BF16, True, True), (2, 32768, 6, F32, F32, True, True), (2, 32768, 4, F32, F32, False, False),
    (300, 64, 4, BF16, BF16, True, False), (601, 8192, 8, BF16, BF16, True, True),
])
def test_norm_matches_definition(T, d, bits, xd, gd, res, smooth):
    x, X = rnd((T, d), 10 * T + d, xd)
    r, R = rnd((T, d), 11 * T + d, xd) if res else (None, None)
    g = np.random.default_rng(5)
    gamma = torch.from_numpy((1 + 0.2 * g.standard_normal(d)).astype(np.float32)).to(gd)
    s_inv = np.exp(g.standard_normal(d)).astype(np.float32) if smooth else None
    H, Y, codes, scales = norm_call(X, R, gamma.cuda(), 1e-6, bits, None if s_inv is None else cuda(s_inv))
    h, rstd, y, near = lowbit.rmsnorm(x, r, gamma.float().numpy(), 1e-6)
    # a statistic this near a border of fp32 (chance about d * 2^-28 a row) would leave rstd's rounding to the
    # order of the sum; the inputs are fixed, and none of their rows is
    assert not near.any()
    if res:
        assert np.array_equal(H.double().cpu().numpy(), rounded(h, xd))
    assert np.array_equal(Y.double().cpu().numpy(), rounded(y, xd))
    v = y if s_inv is None else y * s_inv
    if bits == 4:
        check_mx4(codes, scales, v)
    elif bits != 16:
        q, sa = lowbit.act_codes(v, bits)
        assert np.array_equal(scales.cpu().numpy(), sa)
        assert np.array_equal(codes.cpu().numpy(), q)
        back = torch.empty((T, d), dtype=F32, device="cuda")
        qe.act_dequant(codes, scales, back)
        assert np.array_equal(back.cpu().numpy(), q.astype(np.float32) * sa[:, None])
        b16 = torch.empty((T, d), dtype=BF16, device="cuda")
        qe.act_dequant(codes, scales, b16)
        assert torch.equal(b16, back.to(BF16))


@pytest.mark.parametrize("bits", [8, 4])
def test_norm_rows_that_are_zero_or_not_finite(bits):
    x, X = rnd((6, 512), 7, F32, 0.5)
    X[1] = 0
    X[2, 100] = float("nan")
    X[3, 5] = float("inf")
    X[4, 7] = 3e38          # its square is finite in 64 bits
    g = torch.ones(512, device="cuda")
    _, Y, codes, scales = norm_call(X, None, g, 1e-6, bits, None)
    h, rstd, y, near = lowbit.rmsnorm(X.cpu().numpy(), None, np.ones(512, np.float32), 1e-6)
    assert np.array_equal(Y.cpu().numpy(), y, equal_nan=True)
    if bits == 4:
        check_mx4(codes, scales, y)
    else:
        q, sa = lowbit.act_codes(y, bits)
        assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scales.cpu().numpy(), sa, equal_nan=True)
        assert torch.isnan(scales[2]) and torch.isnan(scales[3]) and scales[1] == 0


def test_norm_in_place():
    x, X = rnd((37, 1536), 8, BF16)
    r, R = rnd((37, 1536), 9, BF16)
    g = torch.ones(1536, dtype=BF16, device="cuda")
    H, Y, codes, scales = norm_call(X, R, g, 1e-6, 8, None)
    X2, R2 = X.clone(), R.clone()
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    qe.add_rmsnorm_quant(X2, g, 1e-6, 8, c2, s2, residual=R2, residual_out=R2, Y=X2)
    assert torch.equal(R2, H) and torch.equal(X2, Y) and torch.equal(c2, codes) and torch.equal(s2, scales)


# ---------------------------------------------------------------- product

def operands(T, K, N, seed, scale_span=None):
    """Random codes on both sides. scale_span e: scale exponents in [-e, e]; None: over the range of trained layers."""
    g = np.random.default_rng(seed)
    out = []
    for rows in (T, N):
        code = g.integers(0, 16, (rows, K)).astype(np.uint8)
        lo, hi = (-12, 4) if scale_span is None else (-scale_span, scale_span)
        scale = (127 + g.integers(lo, hi + 1, (rows, K // 32))).astype(np.uint8)
        # absent rows hold NaN scales: they must reach nothing
        out += [code, scale, cuda(lowbit.pack_codes(code)), cuda(lowbit.tile_scales(scale, 255 if K % 128 == 0 else 127))]
    return out


def product(xc, xs, wc, ws, T, N, dtype):
    guard = torch.full((T * N + 512,), 7.0, dtype=dtype, device="cuda")
    Y = guard[256:256 + T * N].view(T, N)
    if Y.data_ptr() % 16:
        raise AssertionError("the guarded output is not aligned")
    Y.fill_(float("nan"))
    qe.mx4_product(xc, xs, wc, ws, Y)
    torch.cuda.synchronize()
    assert qe.device_error() == 0
    assert (guard[:256] == 7).all() and (guard[256 + T * N:] == 7).all()
    return Y


# T crosses every token tile; N and K leave ragged tiles, scale tiles and half-filled MMAs
SHAPES = [(1, 32, 1), (1, 64, 7), (2, 96, 129), (16, 128, 128), (17, 160, 300), (31, 256, 64), (32, 288, 513), (33, 320, 256),
          (64, 352, 200), (65, 384, 130), (100, 416, 1000), (128, 448, 384), (129, 224, 257), (255, 448, 512), (256, 192, 999),
          (257, 448, 640), (300, 96, 1025), (513, 448, 385), (700, 320, 520), (1100, 448, 777), (300, 64, 1026), (140, 160, 300),
          # K long enough to be split: over clusters of CTAs, of four pairs and of two pairs
          (16, 7264, 300), (40, 1568, 520), (200, 7264, 260), (270, 5120, 514), (1030, 5152, 1000), (513, 6208, 2049),
          # more tiles than pairs of CTAs: with a short K, whose activations are kept, and a longer one
          (2050, 224, 2300), (4900, 1504, 1032), (2310, 1568, 2305)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_exact(T, K, N, dtype):
    """Scale exponents in [-1, 1]: every product is a multiple of 2^-4 and every partial sum at most 36 * 4 * K < 2^20
    (K < 7281), 24 bits in all, so every sum is exact in fp32 whatever its order, and each row and block must meet its own
    scale."""
    x, xe, xc, xs, w, we, wc, ws = operands(T, K, N, T + K + N, 1)
    ref = lowbit.mx4_values(x, xe) @ lowbit.mx4_values(w, we).T
    Y = product(xc, xs, wc, ws, T, N, dtype)
    assert np.array_equal(Y.double().cpu().numpy(), rounded(ref.astype(np.float32), dtype))


@pytest.mark.parametrize("T,K,N", [(1, 8192, 1024), (16, 8960, 1536), (33, 4096, 520), (128, 2080, 384), (200, 8960, 260),
                                   (300, 4128, 513), (520, 1536, 1000), (1030, 2048, 2049), (300, 29568, 264), (1030, 8960, 1000)])
def test_product_long_sums(T, K, N):
    """Wide scales. Products are exact; each of the at most K additions of a sum is off by at most one unit in the last
    place (2^-23) of the magnitudes summed, so |error| <= K * 2^-23 * sum |x w|."""
    x, xe, xc, xs, w, we, wc, ws = operands(T, K, N, T + K + N)
    vx, vw = lowbit.mx4_values(x, xe), lowbit.mx4_values(w, we)
    ref, mag = vx @ vw.T, np.abs(vx) @ np.abs(vw).T
    Y = product(xc, xs, wc, ws, T, N, F32)
    assert (np.abs(Y.double().cpu().numpy() - ref) <= K * 2.0 ** -23 * mag).all()
    again = torch.empty_like(Y)
    qe.mx4_product(xc, xs, wc, ws, again)
    assert torch.equal(again, Y)
    Yb = product(xc, xs, wc, ws, T, N, BF16)
    assert torch.equal(Yb, Y.to(BF16))  # one rounding of the same fp32 sums


@pytest.mark.parametrize("T,N", [(4, 200), (300, 520), (1100, 520)])
def test_product_nan_scales_reach_their_row_and_column_alone(T, N):
    K = 512
    x, xe, xc, xs, w, we, wc, ws = operands(T, K, N, 3, 1)
    xe[T // 2, 5] = 255
    we[N - 1, 15] = 255
    Y = product(xc, cuda(lowbit.tile_scales(xe)), wc, cuda(lowbit.tile_scales(we)), T, N, F32)
    bad = torch.isnan(Y)
    assert bad[T // 2].all() and bad[:, N - 1].all()
    bad[T // 2], bad[:, N - 1] = False, False
    assert not bad.any()


@pytest.mark.parametrize("T,K,N,xd,yd,smooth", [(1, 1536, 256, BF16, BF16, True), (16, 2048, 1000, F32, F32, False),
                                                (130, 1024, 384, BF16, F32, True), (600, 1536, 520, F32, BF16, True)])
def test_linear_layer(T, K, N, xd, yd, smooth):
    x, X = rnd((T, K), 21, xd, 0.5)
    w, W = rnd((N, K), 22, BF16, 0.2)
    s = np.exp(np.random.default_rng(6).standard_normal(K) * 0.5).astype(np.float32) if smooth else None
    layer = qe.Mx4Layer.from_float(W, None if s is None else cuda(s))
    Y = layer.forward(X, out_dtype=yd)
    s_inv = None if s is None else np.float32(1) / s
    vx = lowbit.mx4_values(*lowbit.mx4_quantize(x if s is None else x * s_inv))
    vw = lowbit.mx4_values(*lowbit.mx4_quantize(w if s is None else w * s))
    ref, mag = vx @ vw.T, np.abs(vx) @ np.abs(vw).T
    half = 0.0 if yd == F32 else 2.0 ** -8  # the output's rounding
    assert (np.abs(Y.double().cpu().numpy() - ref) <= K * 2.0 ** -23 * mag * (1 + half) + half * np.abs(ref)).all()
    assert qe.device_error() == 0
    codes, scales = quantize(X, None if s is None else layer.s_inv)
    assert torch.equal(layer.forward_codes(codes, scales, out_dtype=yd), Y)


def test_offsets_beyond_32_bits():
    """Weights whose codes pass 2^32 bytes: the last rows are reached."""
    K, N = 8192, (1 << 20) + 131
    wc = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((qe.mx4_scale_bytes(N, K),), 127, dtype=torch.uint8, device="cuda")
    g = np.random.default_rng(1)
    code = g.integers(0, 16, (140, K)).astype(np.uint8)
    code[:, ::32] = 7  # a 6 in every block, so that quantizing again gives the same codes
    wc[-140:] = cuda(lowbit.pack_codes(code))
    x = g.integers(0, 16, (2, K)).astype(np.uint8)
    xs = np.full((2, K // 32), 127, np.uint8)
    Y = torch.empty((2, N), dtype=F32, device="cuda")
    qe.mx4_product(cuda(lowbit.pack_codes(x)), cuda(lowbit.tile_scales(xs)), wc, ws, Y)
    ref = lowbit.mx4_values(x, xs) @ lowbit.mx4_values(code, np.full((140, K // 32), 127, np.uint8)).T
    # units of 1/4, |sum| <= 36 * 8192 < 2^22: exact
    assert np.array_equal(Y[:, -140:].double().cpu().numpy(), ref) and not Y[:, :-140].any()
    back = torch.empty((N, K), dtype=BF16, device="cuda")
    qe.mx4_dequantize(wc, ws, back)
    codes, scales = torch.zeros_like(wc), torch.zeros_like(ws)
    qe.mx4_quantize(back, codes, scales)
    again = torch.empty((N, K), dtype=BF16, device="cuda")
    qe.mx4_dequantize(codes, scales, again)
    assert torch.equal(again, back) and torch.equal(wc[-140:], codes[-140:])


# ---------------------------------------------------------------- together, as a block uses them

def test_norm_into_mx4_layer():
    T, d, N = 40, 1536, 520
    x, X = rnd((T, d), 31, BF16, 0.5)
    r, R = rnd((T, d), 32, BF16, 0.5)
    w, W = rnd((N, d), 33, BF16, 0.2)
    s = np.exp(np.random.default_rng(7).standard_normal(d) * 0.5).astype(np.float32)
    layer = qe.Mx4Layer.from_float(W, cuda(s))
    g = torch.ones(d, dtype=BF16, device="cuda")
    H, Y, codes, scales = norm_call(X, R, g, 1e-6, 4, layer.s_inv)
    out = layer.forward_codes(codes, scales, out_dtype=F32)
    h, rstd, y, near = lowbit.rmsnorm(x, r, np.ones(d, np.float32), 1e-6)
    assert not near.any()
    vx = lowbit.mx4_values(*lowbit.mx4_quantize(y * (np.float32(1) / s)))
    vw = lowbit.mx4_values(*lowbit.mx4_quantize(w * s))
    assert (np.abs(out.double().cpu().numpy() - vx @ vw.T) <= d * 2.0 ** -23 * (np.abs(vx) @ np.abs(vw).T)).all()


def qe_layer(K, N, a_bits, seed=1):
    g = np.random.default_rng(seed)
    desc = qe.make_desc(K, N, 128 if K % 128 == 0 else 64, 4, a_bits, 8, 4, 4)
    b = lambda *sh: torch.from_numpy((g.standard_normal(sh) * 0.05).astype(np.float32)).to(BF16).cuda()  # noqa: E731
    W, s = b(N, K), cuda(np.exp(g.standard_normal(K) * 0.3).astype(np.float32))
    return qe.QELayer.from_float(desc, W, s, b(K, 8), b(8, N), b(4, K, 4), b(4, 4, N), b(K, 4))


@pytest.mark.parametrize("T", [1, 16, 17, 200, 700])
@pytest.mark.parametrize("a_bits,xd,K", [(8, BF16, 1536), (6, BF16, 320), (8, F32, 1024)])
def test_qe_layer_takes_quantized_rows(T, a_bits, xd, K):
    """With the codes of qe_act_quant, which quantizes as the layer does, the forward is the same bit for bit."""
    layer = qe_layer(K, 392, a_bits)
    x, X = rnd((T, K), 41 + T, xd, 0.5)
    codes, sa = torch.empty((T, K), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    qe.act_quant(X, layer.s_inv, a_bits, codes, sa)
    want = layer.forward(X, out_dtype=F32)
    got = layer.forward_codes(X, codes, sa, out_dtype=F32)
    assert torch.equal(got, want)
    assert qe.device_error() == 0


@pytest.mark.parametrize("bits", [8, 6])
def test_norm_into_qe_layer(bits):
    """The norm's codes through the layer, against the layer's quantization of the norm's row (fp32, so that Y is not
    rounded). The two scales are one unit in the last place apart at most: relative 2^-23. So a code can differ, by one,
    only where v / scale lies within (qmax + 1) * 2^-22 of a half-integer (both quotients' roundings and the scales'
    distance); with the layer's own codes and the norm's, everything behind is the same."""
    T, K = 200, 1536
    layer = qe_layer(K, 392, bits)
    x, X = rnd((T, K), 51, F32, 0.5)
    r, R = rnd((T, K), 52, F32, 0.5)
    g = torch.ones(K, device="cuda")
    H, Y, codes, sa = norm_call(X, R, g, 1e-6, bits, layer.s_inv)
    c2, sa2 = torch.empty_like(codes), torch.empty_like(sa)
    qe.act_quant(Y, layer.s_inv, bits, c2, sa2)
    assert ((sa - sa2).abs() <= sa * 2.0 ** -23).all()
    diff = (codes.int() - c2.int()).cpu()
    assert diff.abs().max() <= 1
    q = ((Y * layer.s_inv).double() / sa.double()[:, None]).cpu()
    assert ((q - q.floor() - 0.5).abs()[diff != 0] <= 2 ** (bits - 1) * 2.0 ** -22).all()
    assert torch.equal(layer.forward_codes(Y, c2, sa2), layer.forward(Y))
    out, own = layer.forward_codes(Y, codes, sa), layer.forward(Y)
    same = (diff == 0).all(1).cuda()
    assert same.any()
    # rows with equal codes: the product's row scales by sa, the adapters' term is the same; three roundings apart
    assert torch.allclose(out[same], own[same], rtol=0, atol=float(own.abs().max()) * 2.0 ** -20)


# ---------------------------------------------------------------- empty calls, streams, graphs

def test_empty_calls():
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    codes, scales = torch.empty((0, 32), dtype=torch.uint8, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")
    qe.mx4_quantize(e, codes, scales)
    qe.mx4_dequantize(codes, scales, e)
    layer = qe.Mx4Layer.from_float(torch.ones((8, 64), dtype=BF16, device="cuda"))
    assert layer.forward(e).shape == (0, 8)
    qe.add_rmsnorm_quant(e, torch.ones(64, dtype=BF16, device="cuda"), 1e-6, 16, Y=e)


@pytest.mark.parametrize("T", [8, 300, 1100])
def test_streams_and_two_calls_at_once(T):
    K, N = 2048, 1024
    w, W = rnd((N, K), 61, BF16, 0.2)
    layer = qe.Mx4Layer.from_float(W)
    xs = [rnd((T, K), 62 + i, BF16)[1] for i in range(2)]
    want = [layer.forward(X) for X in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            got[i].append(layer.forward(xs[i], stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
    raw = layer.forward(xs[0], stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw, want[0])


@pytest.mark.parametrize("T", [1, 16, 200, 1100])
def test_captured_and_replayed(T):
    """A block's norm and product in a graph: replayed on new inputs, also after larger eager calls."""
    d, N = 2048, 1024
    w, W = rnd((N, d), 71, BF16, 0.2)
    layer = qe.Mx4Layer.from_float(W)
    qel = qe_layer(d, 256, 8)
    g = torch.ones(d, dtype=BF16, device="cuda")
    X, R = rnd((T, d), 72, BF16)[1], rnd((T, d), 73, BF16)[1]

    def block(X, R):
        H, Y, codes, scales = norm_call(X, R, g, 1e-6, 4, None)
        H2, Y2, c8, sa = norm_call(X, R, g, 1e-6, 8, qel.s_inv)
        return layer.forward_codes(codes, scales), layer.forward(Y), qel.forward_codes(Y2, c8, sa), H

    block(X, R)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(X, R)
    for seed in (80, 90):
        X.copy_(rnd((T, d), seed, BF16)[1])
        R.copy_(rnd((T, d), seed + 1, BF16)[1])
        layer.forward(rnd((2000, d), 99, BF16)[1])
        want = block(X, R)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert qe.device_error() == 0


def test_binding_refuses_strided_tensors():
    X = torch.zeros((4, 128), dtype=BF16, device="cuda")[:, :64]
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8, device="cuda"), torch.zeros(512, dtype=torch.uint8, device="cuda")
    with pytest.raises(qe.QEError):
        qe.mx4_quantize(X, codes, scales)
    with pytest.raises(qe.QEError):
        qe.add_rmsnorm_quant(X, torch.ones(64, dtype=BF16, device="cuda"), 1e-6, 16, Y=X)


def test_norm_and_layer_agree_with_the_oracle_layer():
    """The whole layer behind the norm, against the C oracle fed with the norm's codes' values."""
    T, K, N = 24, 512, 200
    g = np.random.default_rng(11)
    desc = qe.make_desc(K, N, 128, 4, 8, 0, 1, 0)
    W = torch.from_numpy((g.standard_normal((N, K)) * 0.05).astype(np.float32)).cuda()
    s = np.exp(g.standard_normal(K) * 0.3).astype(np.float32)
    G = torch.zeros((K, 1), dtype=BF16, device="cuda")
    layer = qe.QELayer.from_float(desc, W, cuda(s), None, None, None, None, G)
    x, X = rnd((T, K), 12, F32, 0.5)
    gam = torch.ones(K, device="cuda")
    _, Y, codes, sa = norm_call(X, None, gam, 1e-6, 8, layer.s_inv)
    out = layer.forward_codes(Y, codes, sa)
    wq, wsc, _, _ = oracle.quantize_weights(W.cpu().numpy(), s, 128, 4)
    xv = codes.cpu().numpy().astype(np.float64) * sa.cpu().numpy().astype(np.float64)[:, None]
    wv = np.asarray(wq, np.float64).reshape(N, K // 128, 128) * np.asarray(wsc, np.float64).reshape(N, K // 128)[..., None]
    wv = wv.reshape(N, K)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    # integer group sums are exact; K/128 fp32 multiply-adds and the token scale: (K/128 + 3) half steps
    assert (np.abs(out.double().cpu().numpy() - ref) <= (K // 128 + 3) * 2.0 ** -23 * mag).all()


# ---------------------------------------------------------------- calls the documentation allows and nothing above makes

@pytest.mark.parametrize("bits", [16, 8, 4])
def test_norm_optional_outputs(bits):
    """Every output may be left out; what is written does not change."""
    T, d = 9, 1056
    x, X = rnd((T, d), 91, BF16)
    r, R = rnd((T, d), 92, BF16)
    g = torch.from_numpy(np.random.default_rng(3).standard_normal(d).astype(np.float32)).cuda()
    s = torch.full((d,), 0.5, device="cuda")
    H, Y, codes, scales = norm_call(X, R, g, 1e-5, bits, s)
    for want_y, want_h in ((False, False), (True, False), (False, True)):
        if bits == 16 and not (want_y or want_h):
            continue
        H2, Y2, c2, s2 = norm_call(X, R, g, 1e-5, bits, s, want_y, want_h)
        assert (Y2 is None) == (not want_y) and (Y2 is None or torch.equal(Y2, Y))
        assert (H2 is None) == (not want_h) and (H2 is None or torch.equal(H2, H))
        if bits != 16:
            assert torch.equal(c2, codes) and torch.equal(s2, scales)
    _, y, near = lowbit.rmsnorm(x, r, g.cpu().numpy(), 1e-5)[1:]
    assert not near.any() and np.array_equal(Y.double().cpu().numpy(), rounded(y, BF16))


def at16(t):
    """A copy of t whose address is a multiple of 16 bytes and of no more."""
    n = t.numel() * t.element_size()
    buf = torch.empty(n + 64, dtype=torch.uint8, device="cuda")
    off = (-buf.data_ptr()) % 32 + 16
    c = buf[off:off + n].view(t.dtype).view(t.shape)
    c.copy_(t)
    assert c.data_ptr() % 32 == 16
    return c


@pytest.mark.parametrize("T,K,N", [(5, 1056, 136), (300, 288, 520), (200, 5152, 264)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_least_alignment(T, K, N, dtype):
    x, xe, xc, xs, w, we, wc, ws = operands(T, K, N, 7, 1)
    want = product(xc, xs, wc, ws, T, N, dtype)
    Y = at16(torch.zeros((T, N), dtype=dtype, device="cuda"))
    qe.mx4_product(at16(xc), at16(xs), at16(wc), at16(ws), Y)
    assert torch.equal(Y, want)
    v, V = rnd((T, K), 8, dtype)
    s = at16(torch.full((K,), 0.75, device="cuda"))
    codes, scales = quantize(V, s)
    c2, s2 = at16(torch.zeros_like(codes)), at16(torch.full_like(scales, 0xEE))
    qe.mx4_quantize(at16(V), c2, s2, s=s)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    back, b2 = torch.empty((T, K), dtype=dtype, device="cuda"), at16(torch.zeros((T, K), dtype=dtype, device="cuda"))
    qe.mx4_dequantize(codes, scales, back)
    qe.mx4_dequantize(c2, s2, b2)
    assert torch.equal(b2, back)
    g = torch.ones(K, dtype=dtype, device="cuda")
    H, Yn, c8, sa = norm_call(V, V, g, 1e-6, 8, s)
    Y3, c3, s3 = at16(torch.zeros_like(Yn)), at16(torch.zeros_like(c8)), at16(torch.zeros_like(sa))
    qe.add_rmsnorm_quant(at16(V), at16(g), 1e-6, 8, c3, s3, residual=at16(V), Y=Y3, s_inv=s)
    assert torch.equal(Y3, Yn) and torch.equal(c3, c8) and torch.equal(s3, sa)


def test_very_many_tokens():
    """2^18 + 77 tokens: more token tiles than any group, over every pair of CTAs."""
    T, K, N = (1 << 18) + 77, 64, 40
    g = np.random.default_rng(5)
    code = torch.randint(0, 256, (T, K // 2), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    w = g.integers(0, 16, (N, K)).astype(np.uint8)
    we = np.full((N, 2), 127, np.uint8)
    xs = torch.full((qe.mx4_scale_bytes(T, K),), 128, dtype=torch.uint8, device="cuda")
    Y = product(code, xs, cuda(lowbit.pack_codes(w)), cuda(lowbit.tile_scales(we)), T, N, F32)
    c = code.cpu().numpy()
    x = np.stack((c & 15, c >> 4), -1).reshape(T, K)
    ref = lowbit.mx4_values(x, np.full((T, 2), 128, np.uint8)) @ lowbit.mx4_values(w, we).T
    assert np.array_equal(Y.double().cpu().numpy(), ref)  # multiples of 1/2 below 2^13: exact


@pytest.mark.parametrize("T,N", [(3, 130), (150, 130)])
def test_very_long_rows(T, N):
    """K = 2^20 channels, the longest: the last stages count, and only they hold anything."""
    K, tail = 1 << 20, 4000
    x, xe, xc, xs, w, we, wc, ws = operands(T, tail // 32 * 32, N, 9, 1)
    tail = x.shape[1]

    def place(codes, code, e):
        rows = code.shape[0]
        full = torch.zeros((rows, K // 2), dtype=torch.uint8, device="cuda")
        full[:, (K - tail) // 2:] = codes
        scale = np.full((rows, K // 32), 127, np.uint8)
        scale[:, (K - tail) // 32:] = e
        return full, cuda(lowbit.tile_scales(scale))

    Y = product(*place(xc, x, xe), *place(wc, w, we), T, N, F32)
    ref = lowbit.mx4_values(x, xe) @ lowbit.mx4_values(w, we).T
    assert np.array_equal(Y.double().cpu().numpy(), ref)


def test_many_outputs_with_many_tokens():
    """2^20 + 131 output channels and 150 tokens: only the first and last channels hold anything."""
    T, K, N = 150, 64, (1 << 20) + 131
    x, xe, xc, xs, w, we, wc, ws = operands(T, K, 300, 10, 1)
    full = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    full[:150], full[-150:] = wc[:150], wc[150:]
    scale = np.full((N, K // 32), 127, np.uint8)
    scale[:150], scale[-150:] = we[:150], we[150:]
    Y = product(xc, xs, full, cuda(lowbit.tile_scales(scale)), T, N, BF16)
    ref = rounded((lowbit.mx4_values(x, xe) @ lowbit.mx4_values(w, we).T).astype(np.float32), BF16)
    got = Y.double().cpu().numpy()
    assert np.array_equal(got[:, :150], ref[:, :150]) and np.array_equal(got[:, -150:], ref[:, 150:])
    assert not got[:, 150:-150].any()


def test_weights_quantized_just_before_they_are_used():
    """The linear call may read weights early, but not before the call that writes them: alternating weights in one
    buffer, no synchronization in between."""
    K, N, T = 4096, 4096, 16
    Ws = [rnd((N, K), 95 + i, BF16, 0.2)[1] for i in range(2)]
    X = rnd((T, K), 97, BF16)[1]
    want = [qe.Mx4Layer.from_float(W).forward(X) for W in Ws]
    torch.cuda.synchronize()
    layer = qe.Mx4Layer.from_float(Ws[0])
    got = []
    for i in range(30):
        qe.mx4_quantize(Ws[i % 2], layer.w_codes, layer.w_scales)
        got.append(layer.forward(X))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


def test_activations_written_just_before_they_are_used():
    """Norm, product, and the next norm over the same buffers, back to back, many times: each kernel sees what the one
    before it wrote, and does not overwrite what it still reads."""
    T, d = 64, 2048
    W = rnd((d, d), 98, BF16, 0.2)[1]
    layer = qe.Mx4Layer.from_float(W)
    g = torch.full((d,), 0.7, dtype=BF16, device="cuda")
    codes = torch.empty((T, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty(qe.mx4_scale_bytes(T, d), dtype=torch.uint8, device="cuda")

    def chain(wait):
        h = rnd((T, d), 99, BF16)[1]
        y = h.clone()
        for _ in range(12):
            qe.add_rmsnorm_quant(y, g, 1e-6, 4, codes, scales, residual=h, residual_out=h)
            if wait:
                torch.cuda.synchronize()
            qe.mx4_product(codes, scales, layer.w_codes, layer.w_scales, y)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return h, y

    slow = chain(True)
    for _ in range(5):
        fast = chain(False)
        assert torch.equal(fast[0], slow[0]) and torch.equal(fast[1], slow[1])
    assert torch.isfinite(slow[1]).all()
