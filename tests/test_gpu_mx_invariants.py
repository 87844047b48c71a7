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


# Pieces of 16 bytes a row: every layout of the norm's forward pass, at and beside the widths where it changes.
WIDTHS = [3, 64, 65, 128, 129, 192, 193, 256, 257, 320, 321, 500, 640, 641, 1030, 2048, 2050]


@pytest.mark.parametrize("dt", [BF16, FP32], ids=str)
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("pieces", WIDTHS)
def test_a_norm_s_bits_do_not_depend_on_the_batch(H, pieces, odd, dt):  # noqa: F811
    """A row alone, among few, and among many: the same statistics, norm, codes
    and scales; and the same gradient of the row."""
    hs, m = pieces * (16 // dt.itemsize) - (1 if odd else 0), 700
    say("batches", hs, dt)
    blk, g = H.Block(H.BlockConfig(hc=1, hs=hs, dtype=H.HCGR_BF16 if dt is BF16 else H.HCGR_FP32), 0), gen(hs)
    x = (randn(g, m, hs, scale=3.0) + randn(g, m, 1, scale=8.0)).to(dt)
    w, b, d = randn(g, hs, dtype=dt), randn(g, hs, dtype=dt), randn(g, m, hs, dtype=dt)

    def both(rows):
        return blk.layer_norm(x[rows], w, b, out=blk.alloc_layer_norm(len(x[rows]), quantize=True, keep=True))

    full = both(slice(0, m))
    dx = blk.layer_norm_bwd(x, w, full["stats"], d)["dx"]
    for rows in (slice(0, 1), slice(17, 30), slice(30, 669), slice(60, 700), slice(699, 700)):
        part = both(rows)
        for name in part:
            assert torch.equal(part[name], full[name][rows]), (name, rows)
        got = blk.layer_norm_bwd(x[rows], w, part["stats"], d[rows])["dx"]
        assert torch.equal(got, dx[rows]), rows
