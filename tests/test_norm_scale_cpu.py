"""The library has one int8 quantization of a row: the definition the norm is tested against and the layer's oracle
give the same scales and codes, bit for bit."""
import numpy as np
import pytest

import oracle
from oracle import lowbit


@pytest.mark.parametrize("bits", [8, 6])
def test_norm_definition_quantizes_as_the_layer(bits):
    g = np.random.default_rng(bits)
    v = (g.standard_normal((500, 96)) * np.exp(3 * g.standard_normal((500, 1)))).astype(np.float32)
    v[7] = 0
    codes, sa = lowbit.act_codes(v, bits)
    want, want_sa = oracle.act_quant(v, np.ones(96, np.float32), bits)
    assert np.array_equal(sa, want_sa) and np.array_equal(codes, want)
    # the quotient, rounded once
    qmax = 2 ** (bits - 1) - 1
    assert np.array_equal(sa, (np.abs(v).max(-1).astype(np.float64) / qmax).astype(np.float32))
