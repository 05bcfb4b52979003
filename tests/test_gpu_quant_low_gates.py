"""SwiGLU rows in 8 bits at the low end of the sigmoid's range."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1, 8, 600])
def test_gates_whose_sigmoid_leaves_the_normal_range(cols):
    # The exponential's argument, up to 126 in powers of two, is off by two
    # roundings of 2^-18: 2^-17 ln 2 of the result, the rest a few 2^-24.
    import combine_symmetric_memory_amd as cco
    gates = [-80.0, -86.0, -87.0, -87.25, -87.5, -88.5, -89.0, -100.0, -3e38]
    x = torch.zeros(len(gates), 2 * cols)
    x[:, 0], x[:, cols] = torch.tensor(gates), 2.0 ** 100
    q, s = cco.quant_swiglu(x.cuda())
    want = [g * math.exp(g) / (1.0 + math.exp(g)) * 2.0 ** 100 if g > -87.3 else 0.0
            for g in gates]
    assert q[:, 0].tolist() == [-127 if v else 0 for v in want] and not bool(q[:, 1:].any())
    for got, v in zip(s.tolist(), want):
        assert abs(got * 127 - abs(v)) <= 2.0 ** -17 * abs(v), (got * 127, v)
