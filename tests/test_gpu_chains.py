"""Operators one behind the other on a stream without synchronization, each reading what the one before it is just
writing, against the same chain with a synchronization after every call."""
import pytest
import torch

import quantized_gemm_moe_b200 as qe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def normal(shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * torch.exp(torch.randn((shape[0], 1), generator=g, device="cuda"))).to(dtype)


def agree(chain, times=5):
    """chain(sync) returns its outputs; sync() stands behind every call."""
    slow = chain(torch.cuda.synchronize)
    torch.cuda.synchronize()
    for _ in range(times):
        fast = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(fast, slow))
    assert all(torch.isfinite(t).all() for t in slow)
    assert qe.device_error() == 0


@pytest.mark.parametrize("T,d", [(1, 32), (37, 96), (300, 1536), (2048, 2048)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_norm_and_values_in_turn(T, d, dtype, bits):
    """The norm writes codes and scales that the dequantization behind it reads at once; its values are the next norm's
    input, all in the same buffers. Rows of 32 and 96 channels share cache lines."""
    gamma = torch.full((d,), 0.7, dtype=dtype, device="cuda")
    factor = torch.full((d,), 1.25, device="cuda")

    def chain(sync):
        x, h = normal((T, d), 1, dtype), normal((T, d), 2, dtype)
        if bits == 4:
            codes = torch.empty((T, d // 2), dtype=torch.uint8, device="cuda")
            scales = torch.empty(qe.mx4_scale_bytes(T, d), dtype=torch.uint8, device="cuda")
        else:
            codes, scales = torch.empty((T, d), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        out = []
        for _ in range(12):
            qe.add_rmsnorm_quant(x, gamma, 1e-6, bits, codes, scales, residual=h, residual_out=h, s_inv=factor)
            sync()
            (qe.mx4_dequantize if bits == 4 else qe.act_dequant)(codes, scales, x)
            sync()
            out.append(x.clone())
        return out + [h]

    agree(chain)


@pytest.mark.parametrize("T,d", [(3, 64), (16, 2048), (200, 1024), (1100, 2048)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_and_quantization_in_turn(T, d, dtype):
    """A product's output is quantized at once, with factors that were written just before, and is the next product's input."""
    g = torch.Generator(device="cuda").manual_seed(3)
    W = (torch.randn((d, d), generator=g, device="cuda") * d ** -0.5).to(BF16)
    layer = qe.Mx4Layer.from_float(W)
    gains = [torch.full((d,), f, device="cuda") for f in (0.5, 2.0)]

    def chain(sync):
        y, factor = normal((T, d), 4, dtype), torch.empty(d, device="cuda")
        codes = torch.empty((T, d // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty(qe.mx4_scale_bytes(T, d), dtype=torch.uint8, device="cuda")
        back, out = torch.empty((T, d), dtype=dtype, device="cuda"), []
        for i in range(12):
            factor.copy_(gains[i % 2])
            qe.mx4_quantize(y, codes, scales, s=factor)
            sync()
            qe.mx4_product(codes, scales, layer.w_codes, layer.w_scales, y)
            sync()
            qe.mx4_dequantize(codes, scales, back)
            sync()
            out.append(back.clone())
        return out + [y]

    agree(chain)


def test_values_of_the_largest_rows_and_the_most_tokens():
    """2^20 tokens of 32768 channels, the most the norm writes: 2^32 vectors of eight channels."""
    T, d = 1 << 20, 32768
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 115 << 30:
        pytest.skip("needs 103 GB")
    codes = torch.full((T, d), 3, dtype=torch.int8, device="cuda")
    sa = (torch.arange(T, device="cuda") % 61 + 1).float()
    out = torch.full((T, d), -1.0, dtype=BF16, device="cuda")
    codes[-5:, :] = 1
    qe.act_dequant(codes, sa, out)
    want = 3 * sa  # at most 183: exact in bf16
    want[-5:] = sa[-5:]
    for t in range(0, T, 1 << 14):
        assert (out[t:t + (1 << 14)] == want[t:t + (1 << 14), None]).all()
    del codes, out
    torch.cuda.empty_cache()
