"""The norm's int8 codes are the layer's own: the norm with quantized output in front of the layer gives, bit for bit,
what the layer gives when it quantizes the normed row itself."""
import pytest
import torch

import quantized_gemm_moe_b200 as qe
from test_gpu_lowbit import F32, BF16, norm_call, qe_layer, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 6])
@pytest.mark.parametrize("T,K,gd", [(1, 320, F32), (16, 1536, BF16), (200, 1536, F32), (700, 1024, BF16)])
def test_norm_codes_are_the_layers_own(T, K, gd, bits):
    """Y is fp32 and so not rounded: both quantize the same fl32(y * s_inv)."""
    layer = qe_layer(K, 392, bits)
    X, R = rnd((T, K), 151, F32, 0.5)[1], rnd((T, K), 152, F32, 0.5)[1]
    gamma = (1 + 0.1 * torch.randn(K, generator=torch.Generator().manual_seed(1))).to(gd).cuda()
    H, Y, codes, sa = norm_call(X, R, gamma, 1e-6, bits, layer.s_inv)
    own, own_sa = torch.empty_like(codes), torch.empty_like(sa)
    qe.act_quant(Y, layer.s_inv, bits, own, own_sa)
    assert torch.equal(sa, own_sa) and torch.equal(codes, own)
    assert torch.equal(layer.forward_codes(Y, codes, sa), layer.forward(Y))
    assert qe.device_error() == 0


@pytest.mark.parametrize("bits", [8, 6])
@pytest.mark.parametrize("T,K", [(40, 8), (300, 8960), (5000, 2048), (9, 32768)])
def test_norm_quantizes_as_act_quant(T, K, bits):
    X = rnd((T, K), 153, F32)[1]
    ones = torch.ones(K, device="cuda")
    X[T // 2] = 0
    _, Y, codes, sa = norm_call(X, None, ones, 1e-6, bits, None)
    own, own_sa = torch.empty_like(codes), torch.empty_like(sa)
    qe.act_quant(Y, ones, bits, own, own_sa)
    assert torch.equal(sa, own_sa) and torch.equal(codes, own)
