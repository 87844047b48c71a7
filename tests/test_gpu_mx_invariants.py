"""GPU tests of what the layer norm and the microscaled linear layer promise
beyond each value's bound: where roundings happen, which bits depend on what,
and gradients along the directions that a missing term would show in."""
from __future__ import annotations

import pytest
import torch

import block_reference as B
import mx_reference as X
import norm_directions as N
from test_gpu_block import BF16, DTYPES, EPS, FP16, FP32, H, block, gen, randn, say  # noqa: F401
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


@pytest.mark.parametrize("hs,m", [(33, 7), (67, 5), (1000, 33), (1280, 700), (2560, 9), (2563, 4), (5000, 6), (8192, 4), (24576, 2)])
def test_gradient_along_1_and_h(H, hs, m):  # noqa: F811
    """The kernels' gradient against differences of the kernels' norm, along the
    directions in which a missing term would show (norm_directions)."""
    say("directions", hs, m)
    blk, g = block(H, 1, hs, FP32), gen(hs)
    x = randn(g, m, hs) + 1.0
    w, b = 1 + 0.2 * randn(g, hs).clamp(-3, 3), randn(g, hs)
    d = N.upstream(x, w, randn(g, m, hs))
    stats = blk.layer_norm(x, w, b)["stats"]
    dx = blk.layer_norm_bwd(x, w, stats, d)["dx"]
    N.check(lambda v: blk.layer_norm(v, w, b)["x"], dx, x, w, d, X.layer_norm(x, w, b, EPS)["x"][1],
            X.layer_norm_bwd(x, w, stats, d)["dx"][1], B.C_ROW)


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hs", [1, 8, 67, 504, 1000, 1032, 2048, 2560, 2563, 5000, 8192, 16384, 24576])
def test_norm_of_constant_rows(H, hs, dt):  # noqa: F811
    """Rows of one value v. Where v is a power of two (or zero) every partial sum
    and the mean are exact, so all deviations are 0 and the norm is b, exactly.

    Otherwise a wave's mean is off by at most C*2^-24*|v|, the same in all of its
    values; what it lacks is held to C*2^-24 of itself. So a deviation is off by at
    most 2*(C*2^-24)^2*|v|, times w/sqrt(eps)."""
    say("constant rows", hs, dt)
    blk, g = block(H, 1, hs, dt), gen(hs)
    w, b = (1 + randn(g, hs, scale=0.2)).to(dt), randn(g, hs, dtype=dt)
    for m in (1, 700):
        for v in (0.0, 1.0, -1024.0, 2.0 ** -10, 0.1, -1 / 3, 100.1):
            x = torch.full((m, hs), v, device="cuda").to(dt)
            out = blk.layer_norm(x, w, b)
            if v == 0 or abs(torch.tensor(v)).log2().frac() == 0:
                assert torch.equal(out["x"], b.expand(m, hs)) and bool((out["stats"][:, 0] == v).all()), v
            else:
                slack = 2 * (B.C_ROW * B.U32) ** 2 * float(x[0, 0].double().abs()) / EPS ** 0.5 * w.double().abs()
                B.check(out["x"][:1], (b.double()[None], slack[None] / B.U32), "x", 1)
                assert torch.equal(out["x"], out["x"][:1].expand(m, hs))


# Rows of more than 16384 values, whose scales take the split kernels several turns: the last of them whole and begun,
# each kernel of the product.
DEEP = [(40, 20000, 70), (40, 32768, 20), (4096, 20000, 32), (8192, 16385, 32), (8192, 20000, 64), (1500, 16400, 300), (8192, 20000, 256),
        (2504, 17000, 1200), (2501, 17000, 1000), (2504, 17000, 4000), (2501, 17000, 4000), (10240, 17000, 1400), (10237, 17000, 1400)]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("n,k,m", DEEP)
def test_linear_of_deep_rows(H, n, k, m, dt):  # noqa: F811
    say("deep rows", n, k, m, dt)
    lin, i = linear(H, n, k, dt), linear_inputs(gen(n + k + m), n, k, m, dt, spread=2 if dt is FP16 else 6)
    if dt is FP16:  # sums that fp16 holds
        i["q_scale"] -= 6
    B.check(lin.forward(**i), reference(i, k), "out", X.c_of(k))


# n, k, m and rows of them that take the same kernel with as many waves (held by test_product_choices)
PARTS = [(320, 1000, 61, (3, 19)), (320, 1000, 900, (30, 900)), (10240, 2560, 7, (6, 7)), (10240, 2560, 64, (14, 64)), (1024, 512, 1023, (100, 1000)),
         (2500, 640, 513, (33, 513)), (2500, 640, 4000, (1, 3901)), (10240, 2560, 1400, (77, 1377))]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("n,k,m,rows", PARTS)
def test_a_product_s_rows_are_those_of_a_part_of_the_batch(H, n, k, m, rows, dt):  # noqa: F811
    """Among other rows, in other places of a tile: the same bits."""
    say("part of a batch", n, k, m, rows, dt)
    lin, i = linear(H, n, k, dt), linear_inputs(gen(n + m), n, k, m, dt, spread=2)
    full, (a, z) = lin.forward(**i), rows
    part = lin.forward(i["q"][a:z], i["q_scale"][a:z], i["w"], i["w_scale"], i["bias"])
    assert torch.equal(part.view(torch.uint8), full[a:z].view(torch.uint8))
