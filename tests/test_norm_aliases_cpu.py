"""Which buffers of the norm may be one: residual_out the input or the residual, Y the input, but never both outputs the same
(what is stored second would silently replace the first). Refusals of the C ABI; nothing is launched."""
import pytest

import quantized_gemm_moe_b200 as qe
from test_lowbit_cpu import P, lib, norm  # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_outputs_in_one_buffer_are_refused(lib, bits):  # noqa: F811
    Q = 2 * P
    assert norm(lib, X=P, r=Q, h=P, Y=P, bits=bits, c=3 * P, s=4 * P) == qe.QE_ERR_INVALID_ARG
    assert norm(lib, X=P, r=Q, h=3 * P, Y=3 * P, bits=bits, c=4 * P, s=5 * P) == qe.QE_ERR_INVALID_ARG
    # nothing is written for no rows
    assert norm(lib, X=P, r=Q, h=P, Y=P, T=0, bits=bits) == qe.QE_OK
