"""The example's block with all of its gradients, in both layouts, against plain torch in fp32.

Tolerance: 8-bit rounding.  E4M3 keeps 4 significant bits: a relative error of up to 2^-4, 2.6% in the mean square, for each
cast that a gradient passes.  Twice the square root of their number, as the activation's derivative may double one:
down: the first product's two operands and the second's (3); router: the second's weights too (4); up: the cast of the
gradient, the transposed weights, the first product's two operands and the checkpoint (5), and the operand itself (6);
input and norm: 5, the cast that is carried on, the transposed weights (7) and what passes the router, whose part is the
smaller.  Capacities: at most 256 rows an expert, so that no slot is dropped.
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

CASTS = dict(ddown=3, drouter=4, dup=6, dx=7, dnorm=7)


@pytest.mark.parametrize("tokens,decode", [(700, False), (40, True), (1, True), (1, False), (129, False)])
def test_gradients(tokens, decode):
    found = moe_layer.main(["--train", "--tokens", str(tokens), "--hidden", "1024", "--inner", "512"]
                           + ["--decode"] * decode)
    for name, casts in CASTS.items():
        assert found[name] < 2 * casts ** 0.5 * 0.026, name
