"""CPU checks of the norm / MXFP4 entry points: the oracle's definitions against hand-worked cases, sizes,
and the refusals of the C ABI and of the binding. Nothing is launched."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_gemm_moe_b200 as qe
from oracle import lowbit

OK, BAD, UNSUP, ALIGN, WS = (qe.QE_OK, qe.QE_ERR_INVALID_ARG, qe.QE_ERR_UNSUPPORTED, qe.QE_ERR_ALIGNMENT,
                             qe.QE_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    from quantized_gemm_moe_b200 import build
    build.build()
    return qe.load()


# ---------------------------------------------------------------- the oracle

def test_oracle_codes_ties_and_saturation():
    v = np.zeros((1, 32), np.float32)
    v[0, :15] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5, -0.3, -0.0, 0.26, 4.99, 5.01, -6.0, 4.0]
    code, scale = lowbit.mx4_quantize(v)
    # max 7.5 = 1.875 * 2^2: E = 0, so the values stay as they are
    assert scale[0, 0] == 127
    want = [0, 1, 1, 2, 2, 4, 4, 6, -0.5, 0, 0.5, 4, 6, -6, 4]
    assert np.array_equal(lowbit.mx4_values(code, scale)[0, :15], want)
    assert code[0, 9] == 8  # the sign of a negative zero is kept


@pytest.mark.parametrize("top,E", [(4.0, 0), (7.99, 0), (8.0, 1), (3.99, -1), (1.0, -2), (3.4e38, 125), (2.0 ** -124, -126),
                                   (2.0 ** -126, -127), (1e-44, -127), (0.0, -127)])
def test_oracle_scale_exponent(top, E):
    v = np.zeros((1, 64), np.float32)
    v[0, 5] = top
    _, scale = lowbit.mx4_quantize(v)
    assert scale[0, 0] == E + 127 and scale[0, 1] == 0


def test_oracle_values_on_the_grid_survive():
    g = np.random.default_rng(1)
    code = g.integers(0, 16, (40, 96)).astype(np.uint8)
    code[:, ::32] = 7  # a 6 in every block fixes its exponent
    scale = g.integers(10, 240, (40, 3)).astype(np.uint8)
    v = lowbit.mx4_values(code, scale).astype(np.float32)
    c, s = lowbit.mx4_quantize(v)
    assert np.array_equal(s, scale) and np.array_equal(c, code)


def test_oracle_block_that_is_not_finite():
    v = np.ones((1, 96), np.float32)
    v[0, 3], v[0, 40] = np.nan, np.inf
    code, scale = lowbit.mx4_quantize(v)
    assert list(scale[0]) == [255, 255, 125] and not code[0, :64].any() and (code[0, 64:] == 6).all()


def test_oracle_scale_tiles():
    off = lowbit.scale_offsets(300, 288)
    assert off[0, 0] == 0 and off[1, 0] == 16 and off[32, 0] == 4 and off[0, 3] == 3 and off[0, 4] == 512
    assert off[128, 0] == 3 * 512 and off[299, 8] == (2 * 3 + 2) * 512 + (299 % 32) * 16 + (299 % 128) // 32 * 4
    assert len(np.unique(off)) == off.size and off.max() < 3 * 3 * 512


def test_oracle_rmsnorm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]], np.float32)
    h, rstd, y, _ = lowbit.rmsnorm(x, x, np.full(8, 2.0, np.float32), 0.0)
    assert np.array_equal(h, 2 * x)
    assert rstd[0] == np.float32(1 / np.sqrt(100 / 8)) and y[0, 0] == np.float32(np.float32(6 * rstd[0]) * 2)
    q, sa = lowbit.act_codes(np.array([[1.0, -2.0, 0.5]], np.float32), 6)
    assert sa[0] == np.float32(2) * np.float32(1 / 31) and list(q[0]) == [16, -31, 8]  # 15.5 and 7.75: to even, to nearest
    q, sa = lowbit.act_codes(np.array([[1.0, np.inf], [0.0, 0.0]], np.float32), 8)
    assert np.isnan(sa[0]) and sa[1] == 0 and not q.any()


# ---------------------------------------------------------------- sizes

def test_sizes(lib):
    assert qe.mx4_code_bytes(3, 96) == 144 and qe.mx4_code_bytes(0, 32) == 0
    assert qe.mx4_scale_bytes(1, 32) == 512 and qe.mx4_scale_bytes(129, 160) == 4 * 512
    assert qe.mx4_scale_bytes(29568, 8192) == 231 * 64 * 512
    assert qe.mx4_linear_workspace_bytes(16, 8192) == 16 * 4096 + 64 * 512
    assert qe.mx4_linear_workspace_bytes(1, 32) == 256 + 512
    # 64-bit sizes: 2^24 rows of 2^20 channels
    assert qe.mx4_code_bytes(1 << 24, 1 << 20) == 1 << 43
    for rows, cols in ((-1, 32), (1, 0), (1, 33), (1, 48), ((1 << 24) + 1, 32), (1, (1 << 20) + 32)):
        assert qe.mx4_code_bytes(rows, cols) == 0 and qe.mx4_scale_bytes(rows, cols) == 0
    assert qe.mx4_linear_workspace_bytes(-1, 64) == 0 and qe.mx4_linear_workspace_bytes(4, 65) == 0


# ---------------------------------------------------------------- refusals of the C ABI (pointers are never read)

P = 4096  # an aligned address nothing is launched on


def norm(lib, **k):
    a = dict(X=P, xd=1, r=None, g=P, gd=1, eps=1e-6, T=4, d=64, si=None, bits=8, h=None, Y=P, c=P, s=P)
    a.update(k)
    return lib.qe_add_rmsnorm_quant(a["X"], a["xd"], a["r"], a["g"], a["gd"], a["eps"], a["T"], a["d"], a["si"], a["bits"],
                                    a["h"], a["Y"], a["c"], a["s"], None)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), OK), (dict(T=0, X=None, c=None, s=None, Y=None), OK),
    (dict(T=-1), BAD), (dict(T=(1 << 20) + 1), BAD), (dict(d=0), BAD), (dict(d=60), UNSUP), (dict(bits=4, d=72), UNSUP),
    (dict(d=32776), UNSUP), (dict(bits=5), UNSUP), (dict(xd=2), BAD), (dict(gd=-1), BAD), (dict(eps=-1e-9), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(X=None), BAD), (dict(g=None), BAD), (dict(c=None), BAD),
    (dict(s=None), BAD), (dict(h=P), BAD), (dict(bits=16, Y=None), BAD), (dict(X=P + 2), ALIGN), (dict(Y=P + 8), ALIGN),
    (dict(c=P + 4), ALIGN), (dict(si=P + 4), ALIGN), (dict(r=P + 8), ALIGN), (dict(r=P, h=P + 8), ALIGN), (dict(s=P + 8), ALIGN),
])
def test_norm_refusals(lib, change, status):
    assert norm(lib, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), OK), (dict(rows=-1), BAD), (dict(cols=31), BAD), (dict(cols=0), BAD), (dict(rows=(1 << 24) + 1), UNSUP),
    (dict(cols=(1 << 20) + 32), UNSUP), (dict(xd=5), BAD), (dict(X=None), BAD), (dict(c=None), BAD), (dict(sc=None), BAD),
    (dict(si=P), BAD), (dict(X=P + 2), ALIGN), (dict(c=P + 8), ALIGN), (dict(sc=P + 4), ALIGN), (dict(s=P + 4), ALIGN),
    (dict(s=P, si=P + 4), ALIGN),
])
def test_quantize_refusals(lib, change, status):
    a = dict(X=P, xd=1, s=None, rows=4, cols=64, c=P, sc=P, si=None)
    a.update(change)
    assert lib.qe_mx4_quantize(a["X"], a["xd"], a["s"], a["rows"], a["cols"], a["c"], a["sc"], a["si"], None) == status
    if "s" not in change and "si" not in change:
        assert lib.qe_mx4_dequantize(a["c"], a["sc"], a["rows"], a["cols"], a["X"], a["xd"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=0), OK), (dict(T=0, x=None, xs=None, Y=None), OK), (dict(T=-1), BAD), (dict(T=(1 << 20) + 1), BAD), (dict(K=40), BAD),
    (dict(K=0), BAD), (dict(N=0), BAD), (dict(N=(1 << 24) + 1), UNSUP), (dict(K=(1 << 20) + 32), UNSUP), (dict(yd=3), BAD),
    (dict(w=None), BAD), (dict(ws=None), BAD), (dict(x=None), BAD), (dict(xs=None), BAD), (dict(Y=None), BAD), (dict(x=P + 8), ALIGN),
    (dict(xs=P + 8), ALIGN), (dict(w=P + 8), ALIGN), (dict(ws=P + 8), ALIGN), (dict(Y=P + 8), ALIGN),
])
def test_product_refusals(lib, change, status):
    a = dict(x=P, xs=P, w=P, ws=P, T=4, K=64, N=8, Y=P, yd=1)
    a.update(change)
    assert lib.qe_mx4_product(a["x"], a["xs"], a["w"], a["ws"], a["T"], a["K"], a["N"], a["Y"], a["yd"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=0), OK), (dict(T=0, X=None, work=None), OK), (dict(T=-1), BAD), (dict(K=40), BAD), (dict(xd=2), BAD), (dict(yd=2), BAD),
    (dict(w=None), BAD), (dict(X=None), BAD), (dict(X=P + 8), ALIGN), (dict(si=P + 8), ALIGN), (dict(work=None), WS),
    (dict(nbytes=767), WS), (dict(work=P + 8), ALIGN),
])
def test_linear_refusals(lib, change, status):
    a = dict(w=P, ws=P, si=None, X=P, xd=1, T=4, K=64, N=8, Y=P, yd=1, work=P, nbytes=768)
    a.update(change)
    assert qe.mx4_linear_workspace_bytes(4, 64) == 768
    assert lib.qe_mx4_linear_forward(a["w"], a["ws"], a["si"], a["X"], a["xd"], a["T"], a["K"], a["N"], a["Y"], a["yd"], a["work"],
                                     a["nbytes"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=0), OK), (dict(a_bits=16), UNSUP), (dict(c=None), BAD), (dict(sa=None), BAD), (dict(c=P + 8), ALIGN),
    (dict(sa=P + 8), ALIGN), (dict(X=None), BAD), (dict(T=-1), BAD), (dict(work=None), WS),
])
def test_forward_codes_refusals(lib, change, status):
    a = dict(a_bits=8, X=P, c=P, sa=P, T=4, work=P)
    a.update(change)
    d = qe.make_desc(256, 256, 64, 4, a["a_bits"], 8, 4, 4)
    w = qe.LayerWeights(P, P, P, P)
    assert lib.qe_linear_forward_codes(ctypes.byref(d), ctypes.byref(w), a["X"], 0, a["c"], a["sa"], a["T"], P, 0, a["work"],
                                       1 << 30, None) == status


@pytest.mark.parametrize("change,status", [(dict(T=0), OK), (dict(T=-1), BAD), (dict(d=12), UNSUP), (dict(od=2), BAD),
                                           (dict(c=None), BAD), (dict(sa=None), BAD), (dict(o=None), BAD), (dict(c=P + 8), ALIGN)])
def test_act_dequant_refusals(lib, change, status):
    a = dict(c=P, sa=P, T=2, d=64, o=P, od=1)
    a.update(change)
    assert lib.qe_act_dequant(a["c"], a["sa"], a["T"], a["d"], a["o"], a["od"], None) == status


# ---------------------------------------------------------------- refusals of the binding (CPU tensors reach no launch)

def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    X = torch.zeros(4, 64, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    Y = torch.zeros(4, 8, dtype=torch.bfloat16)
    wc, wsc = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)

    def refused(f, *a, **k):
        with pytest.raises(qe.QEError) as e:
            f(*a, **k)
        assert e.value.status == BAD

    refused(qe.mx4_quantize, X, codes, scales)                       # not on a GPU
    refused(qe.mx4_quantize, X, codes[:, :31], scales)
    refused(qe.mx4_quantize, X, codes, scales[:511])
    refused(qe.mx4_quantize, X[0], codes, scales)
    refused(qe.mx4_quantize, X.half(), codes, scales)
    refused(qe.mx4_quantize, X, codes, scales, s=torch.ones(63))
    refused(qe.mx4_dequantize, codes, scales, X[:3])
    refused(qe.mx4_product, codes, scales, wc, wsc, Y)
    refused(qe.mx4_product, codes[:3], scales, wc, wsc, Y)
    refused(qe.mx4_product, codes, scales, wc[:7], wsc, Y)
    refused(qe.mx4_linear_forward, wc, wsc, X, Y, scales)
    refused(qe.mx4_linear_forward, wc, wsc, X, Y[:3], scales)
    g = torch.ones(64, dtype=torch.bfloat16)
    i8, sa = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    refused(qe.add_rmsnorm_quant, X, g, 1e-6, 8, i8, sa)
    refused(qe.add_rmsnorm_quant, X, g[:63], 1e-6, 8, i8, sa)
    refused(qe.add_rmsnorm_quant, X, g, 1e-6, 8, codes, sa)          # MXFP4 codes for int8
    refused(qe.add_rmsnorm_quant, X, g, 1e-6, 4, i8, scales)
    refused(qe.add_rmsnorm_quant, X, g, 1e-6, 8, i8, sa, residual=X.float())
    refused(qe.act_dequant, i8, sa[:3], X)
