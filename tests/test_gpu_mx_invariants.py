"""GPU tests of what the layer norm and the microscaled linear layer promise
beyond each value's bound: where roundings happen, which bits depend on what,
and gradients along the directions that a missing term would show in."""
from __future__ import annotations

import pytest
import torch

import block_reference as B
import mx_reference as X
from test_gpu_block import BF16, FP16, FP32, H, gen, randn, say  # noqa: F401
from test_gpu_mx import linear, linear_inputs, reference

pytestmark = pytest.mark.gpu


# A shape for each kernel of the product (16 x 16 to 64 x 64 split, tiles of 128 x 128, 192 x 256 and 256 x 256 with
# and without whole pieces of output).
BIAS = [(200, 300, 1), (4096, 2560, 32), (1024, 512, 1023), (2563, 2560, 190), (2560, 10240, 512), (2500, 640, 513), (2501, 640, 513),
        (2500, 640, 4000), (2501, 640, 4000), (10240, 2560, 1400), (10237, 2560, 1400)]


@pytest.mark.parametrize("n,k,m", BIAS)
def test_bias_joins_the_whole_sum(H, n, k, m):  # noqa: F811
    """A bias of 2^20 next to sums of some 2^4: the result is the sum, off by its
    own roundings, and the bias, rounded once. (Roundings of partial sums at the
    bias's size would be half steps of 2^-3 each.)"""
    say("large bias", n, k, m)
    lin, i = linear(H, n, k, FP32), linear_inputs(gen(n + m), n, k, m, FP32, spread=2)
    i["bias"] = randn(gen(m), n, scale=2.0 ** 20)
    val, amp = X.linear(i["q"], i["q_scale"], i["w"], i["w_scale"], None, k)
    B.check(lin.forward(**i), (val + i["bias"].double(), amp), "out", X.c_of(k))
