"""The example layer, forward and backward, in both 8-bit formats and layouts, against plain torch in fp32.

Tolerance: 8-bit rounding.  A uniform rounding error of half a code is 2^-8 / sqrt(3) of the largest value for int8 (rows of
~1000 normal values: largest about 3.5 sigma, so 0.8% of sigma), and E4M3 keeps 4 significant bits (relative error up to
2^-4, 2.6% in the mean square).  Four roundings meet (two operands, two products), the second pair through a product of
two factors: under 2 sqrt(4) times one, 3.2% and 10.4%.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import moe_layer  # noqa: E402


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("decode", [False, True])
def test_layer(int8, decode):
    found = moe_layer.main(["--train", "--tokens", "40" if decode else "700", "--hidden", "1024", "--inner", "512"]
                           + ["--int8"] * int8 + ["--decode"] * decode)
    bound = 0.032 if int8 else 0.104
    assert found["out"] < bound and found["dlogits"] < bound
