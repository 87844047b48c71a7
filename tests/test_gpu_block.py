"""GPU tests of the block operators (the norms around a block and their
gradients, the row quantizer, the 8-bit linear layer) against the 64-bit
reference, at the widths, lengths, strides and values where they can go wrong."""
from __future__ import annotations

import pytest
import torch

import block_reference as B

pytestmark = pytest.mark.gpu

EPS, RHO = 1e-6, 0.75
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def H():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import skinny_gemm_hcgr_amd as H
    H.load_library()
    return H


def code(H, dt):
    return {BF16: H.HCGR_BF16, FP16: H.HCGR_FP16, FP32: H.HCGR_FP32}[dt]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=FP32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def say(*a):
    print("[block]", *a, flush=True)


def block(H, hc, hs, dt, **kw):
    return H.Block(H.BlockConfig(hc=hc, hs=hs, dtype=code(H, dt), **{"eps": EPS, "res_scale": RHO, **kw}), 0)


# widths: one value, odd ones (no 16-byte pieces), one wave, several waves,
# whole and ragged 16-byte pieces, wider than one workgroup's registers
WIDTHS = [1, 3, 8, 67, 128, 504, 520, 1000, 2560, 4100, 10240, 24576]
LENGTHS = {1: (1, 5), 3: (2,), 8: (1, 300), 67: (1, 33), 128: (1, 4, 1030), 504: (3, 513), 520: (2, 7),
           1000: (1, 333), 2560: (1, 2, 16, 700), 4100: (3, 65), 10240: (1, 9), 24576: (2,)}
SHAPES = [(hs, m) for hs in WIDTHS for m in LENGTHS[hs]]
DTYPES = [BF16, FP16, FP32]


# -------------------------------------------------------------------- norm --
@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hs,m", SHAPES)
def test_norm(H, hs, m, dt):
    say("norm", hs, m, dt)
    g = gen(hs + m)
    blk = block(H, 1, hs, dt)
    x, w = randn(g, m, hs, dtype=dt, scale=3.0), randn(g, hs, dtype=dt, scale=0.2)
    ref = B.norm(x, w, EPS)
    out = blk.norm(x, w)
    B.check(out["x"], ref["x"], "x")
    B.check(out["rrms"], ref["rrms"], "rrms")
    both = blk.norm(x, w, out=blk.alloc_norm(m, quantize=True, keep=True))
    assert torch.equal(both["x"], out["x"]) and torch.equal(both["rrms"], out["rrms"])
    B.check_quantized(both["q"], both["q_scale"], *ref["x"], "q")
    only = blk.norm(x, w, quantize=True)
    assert "x" not in only and torch.equal(only["q"], both["q"]) and torch.equal(only["q_scale"], both["q_scale"])


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hs,m", SHAPES)
def test_norm_bwd(H, hs, m, dt):
    say("norm_bwd", hs, m, dt)
    g = gen(hs + m + 1)
    blk = block(H, 1, hs, dt)
    x, w, d = (randn(g, m, hs, dtype=dt, scale=3.0), randn(g, hs, dtype=dt, scale=0.2), randn(g, m, hs, dtype=dt))
    rrms = blk.norm(x, w)["rrms"]
    ref = B.norm_bwd(x, w, rrms, d)
    out = blk.norm_bwd(x, w, rrms, d)
    B.check(out["dx"], ref["dx"], "dx")
    B.check(out["dw"], ref["dw"], "dw", B.C_ROW + m)
    for keep in ("dx", "dw"):  # each gradient alone
        one = blk.norm_bwd(x, w, rrms, d, out={keep: torch.empty_like(out[keep])})
        assert torch.equal(one[keep], out[keep]), keep


# ---------------------------------------------------------------- residual --
def residual_inputs(g, m, hc, hs, dt, gates=True, post=True, pre=True):
    return {"R": randn(g, m, hc * hs, dtype=dt, scale=2.0), "y": randn(g, m, hs, dtype=dt, scale=3.0),
            "inj": randn(g, m, hc, dtype=dt, scale=2.0) if gates else None,
            "w_post": randn(g, hs, dtype=dt, scale=0.2) if post else None,
            "w_pre": randn(g, hs, dtype=dt, scale=0.2) if pre else None}


def check_residual(out, ref, pre, post):
    B.check(out["R2"], ref["R2"], "R2")
    if post:
        B.check(out["rrms"][:, 0], (ref["rrms"][0],) * 2, "rrms of the norm after")
    if pre:
        # r of a sum that may cancel: its terms' sizes count, as in x
        B.check(out["rrms"][:, 1], (ref["rrms"][1], ref["rrms"][1] * amplification(ref)), "rrms of the next norm")
        if "x" in out:
            B.check(out["x"], ref["x"], "x", B.C_ROW * amplification(ref)[:, None])


def amplification(ref):
    """How much larger the terms of u are than u itself, in the row's RMS."""
    v, a = ref["x"]
    return ((a * a).mean(1) / (v * v).mean(1)).sqrt().clamp(min=1.0)


RES_SHAPES = [(hc, hs, m) for hc, hs, m in [
    (1, 1, 3), (2, 3, 5), (8, 8, 2), (4, 67, 33), (1, 128, 1030), (4, 128, 5), (2, 504, 513), (8, 520, 7), (2, 1000, 333),
    (4, 2560, 1), (4, 2560, 16), (4, 2560, 700), (8, 2560, 9), (1, 2560, 64), (2, 4100, 65), (4, 10240, 3),
    (8, 10240, 2), (1, 24576, 2), (8, 24576, 2), (8, 8192, 5), (8, 8187, 3), (4, 8192, 300), (2, 2563, 900),
    (4, 517, 1700), (8, 16384, 2)]]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hc,hs,m", RES_SHAPES)
def test_residual(H, hc, hs, m, dt):
    say("residual", hc, hs, m, dt)
    blk = block(H, hc, hs, dt)
    i = residual_inputs(gen(hs + m + hc), m, hc, hs, dt)
    ref = B.residual(**i, hc=hc, eps=EPS, rho=RHO)
    out = blk.residual(**i)
    check_residual(out, ref, True, True)
    both = blk.residual(**i, out=blk.alloc_residual(m, quantize=True, keep=True))
    for k in ("R2", "x", "rrms"):
        assert torch.equal(both[k], out[k]), k
    B.check_quantized(both["q"], both["q_scale"], *ref["x"], "q",
                      B.C_ROW * float(amplification(ref).max()))


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hc,hs,m", RES_SHAPES)
def test_residual_bwd(H, hc, hs, m, dt):
    say("residual_bwd", hc, hs, m, dt)
    blk = block(H, hc, hs, dt)
    g = gen(hs + m + hc + 1)
    i = residual_inputs(g, m, hc, hs, dt)
    rrms = blk.residual(**i)["rrms"]
    d = {"dR2": randn(g, m, hc * hs, dtype=dt), "dx": randn(g, m, hs, dtype=dt)}
    ref = B.residual_bwd(**i, rrms=rrms, **d, hc=hc, rho=RHO)
    out = blk.residual_bwd(**i, rrms=rrms, **d)
    assert set(out) == set(ref)
    for k in ref:
        B.check(out[k], ref[k], k, B.C_ROW + (m if k.startswith("dw") else 0))


@pytest.mark.parametrize("hc,hs,m", [(1, 1000, 5), (4, 2560, 3), (2, 67, 9), (4, 24576, 2)])
@pytest.mark.parametrize("gates,post,pre,from_R2", [(0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (0, 0, 0, 1), (1, 1, 1, 0),
                                                    (0, 0, 1, 0)])
def test_residual_parts(H, hc, hs, m, gates, post, pre, from_R2):
    """Each optional part left out, forward and backward."""
    say("parts", hc, hs, m, gates, post, pre, from_R2)
    blk, g = block(H, hc, hs, BF16), gen(hc * hs)
    i = residual_inputs(g, m, hc, hs, BF16, gates, post, pre)
    ref = B.residual(**i, hc=hc, eps=EPS, rho=RHO)
    out = blk.residual(**i)
    check_residual(out, ref, pre, post)
    rrms = out["rrms"] if pre or post else None
    d = {"dR2": randn(g, m, hc * hs, dtype=BF16) if from_R2 else None,
         "dx": randn(g, m, hs, dtype=BF16) if pre else None}
    want = B.residual_bwd(**i, rrms=rrms, **d, hc=hc, rho=RHO)
    got = blk.residual_bwd(**i, rrms=rrms, **d)
    assert set(got) == set(want)
    for k in want:
        B.check(got[k], want[k], k, B.C_ROW + (m if k.startswith("dw") else 0))


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hc,hs", [(1, 1), (2, 8), (4, 100), (4, 2560), (8, 2560), (2, 40000)])
def test_gradient_of_gates_far_from_zero(H, hc, hs, dt):
    """inj/HC up to +-20, z and dR2 positive, so that the sum's terms do not
    cancel and the bound is relative to the gradient itself. For large positive
    logits the slope of the gate is far below the gate's own rounding."""
    say("gates", hc, hs, dt)
    steps = torch.tensor([-20.0, -16, -12, -8, -3, 0, 3, 8, 12, 16, 20], device="cuda")
    m, g = len(steps), gen(hc + hs)
    inj = (torch.stack([steps.roll(s) for s in range(hc)], 1) * hc).to(dt)  # all of them exact in 8 bits
    assert torch.equal(inj.float(), torch.stack([steps.roll(s) for s in range(hc)], 1) * hc)
    scale = 1.0 if dt is not FP16 else 2.0 ** 14 / hs  # sums that keep slope * sum a normal number of 16 bits
    y, dR2 = (0.5 + torch.rand(m, k, generator=g, device="cuda") for k in (hs, hc * hs))
    i = {"R": randn(g, m, hc * hs, dtype=dt), "y": y.to(dt), "inj": inj, "w_post": None, "w_pre": None}
    d = {"dR2": (dR2 * scale).to(dt), "dx": None}
    ref = B.residual_bwd(**i, rrms=None, **d, hc=hc, rho=RHO)
    got = block(H, hc, hs, dt).residual_bwd(**i, rrms=None, **d)
    B.check(got["dinj"], ref["dinj"], "dinj")
    B.check(got["dy"], ref["dy"], "dy")


def test_plain_combine_is_the_op_s_combine(H):
    """Without norms and with a residual scale of 1 the operator is COMBINE."""
    m, hc, hs = 50, 4, 2560
    i = residual_inputs(gen(7), m, hc, hs, BF16, post=False, pre=False)
    out = block(H, hc, hs, BF16, res_scale=1.0).residual(**i)["R2"]
    op = H.HCGR(H.Config(hc=hc, hs=hs), 0)
    ref = op.combine(i["R"], i["y"], i["inj"])
    # both within half a step of the same value (plus 32-bit roundings): at most a step apart
    d = (out.double() - ref.double()).abs()
    assert bool((d <= torch.finfo(BF16).eps * ref.double().abs() + 2.0 ** -20).all())
    assert float((d > 0).float().mean()) < 1e-3


# Shapes of the kernels that the lists above do not reach (test_block_launches.py
# checks that every kernel is reached): wide rows of odd widths, by passes or two
# pieces a thread, and wide rows of one and two streams.
OTHER_NORM = [(1001, 9), (2563, 5), (4096, 6), (8187, 4), (8192, 5), (9001, 3), (16383, 3), (24577, 3), (65535, 2)]
OTHER_RES = [(8, 1001, 6), (8, 2563, 3), (4, 2563, 5), (4, 8187, 3), (1, 2563, 40), (1, 8192, 5), (2, 8192, 5),
             (2, 4096, 7), (1, 16384, 2), (2, 16384, 3), (1, 8187, 3), (2, 24577, 2), (4, 9001, 2)]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hs,m", OTHER_NORM)
def test_norm_of_other_widths(H, hs, m, dt):
    test_norm(H, hs, m, dt)
    test_norm_bwd(H, hs, m, dt)
    test_quantize(H, hs, m, dt)


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("hc,hs,m", OTHER_RES)
def test_residual_of_other_widths(H, hc, hs, m, dt):
    test_residual(H, hc, hs, m, dt)
    test_residual_bwd(H, hc, hs, m, dt)


# ------------------------------------------------- strides, streams, graphs --
@pytest.mark.parametrize("hs,off", [(2560, 0), (2560, 1), (1000, 8), (129, 0)])
def test_strided_and_unaligned_rows(H, hs, off):
    """Rows inside wider tensors, aligned to 16 bytes or not, give the bits of
    dense rows; what lies around strided outputs stays."""
    m, hc, dt = 37, 2, BF16
    say("strided", hs, off)
    blk, g = block(H, hc, hs, dt), gen(3)
    i = residual_inputs(g, m, hc, hs, dt)
    wide = torch.full((m, hs + 24), float("nan"), dtype=dt, device="cuda")
    wide[:, off:off + hs] = i["y"]
    winj = torch.full((m, hc + 3), float("nan"), dtype=dt, device="cuda")
    winj[:, 1:1 + hc] = i["inj"]
    want = blk.residual(**i)
    got = blk.residual(i["R"], wide[:, off:off + hs], winj[:, 1:1 + hc], i["w_post"], i["w_pre"])
    ref = B.residual(**i, hc=hc, eps=EPS, rho=RHO)
    check_residual(got, ref, True, True)
    if off % 8 == 0 and hs % 8 == 0:
        assert all(torch.equal(got[k], want[k]) for k in want)
    n = block(H, 1, hs, dt)
    B.check(n.norm(wide[:, off:off + hs], i["w_pre"])["x"], B.norm(i["y"], i["w_pre"], EPS)["x"], "x")
    dR2, dx = randn(g, m, hc * hs, dtype=dt), randn(g, m, hs, dtype=dt)
    out = blk.alloc_residual_bwd(m)
    around = torch.full((m, hc + 3), 5.0, dtype=dt, device="cuda")
    out["dinj"] = around[:, 1:1 + hc]
    got = blk.residual_bwd(i["R"], wide[:, off:off + hs], winj[:, 1:1 + hc], i["w_post"], i["w_pre"], want["rrms"], dR2,
                           dx, out=out)
    ref = B.residual_bwd(**i, rrms=want["rrms"], dR2=dR2, dx=dx, hc=hc, rho=RHO)
    for k in ref:
        B.check(got[k], ref[k], k, B.C_ROW + (m if k.startswith("dw") else 0))
    assert bool((around[:, 0] == 5).all()) and bool((around[:, 1 + hc:] == 5).all())


@pytest.mark.parametrize("hs", [40, 67, 2560])
def test_quantized_rows_leave_their_padding(H, hs):
    m, ld = 21, (hs + 15) // 16 * 16 + 32
    blk, g = block(H, 1, hs, BF16), gen(4)
    x, w = randn(g, m, hs, dtype=BF16), randn(g, hs, dtype=BF16, scale=0.1)
    buf = torch.full((m + 2, ld), 77, dtype=torch.int8, device="cuda")
    out = {"q": buf[:m, :hs], "q_scale": torch.empty(m, device="cuda")}
    blk.norm(x, w, out=out)
    B.check_quantized(out["q"], out["q_scale"], *B.norm(x, w, EPS)["x"], "q")
    assert bool((buf[:, hs:] == 77).all()) and bool((buf[m:] == 77).all())


def test_empty_batch(H):
    blk = block(H, 4, 256, BF16)
    w = torch.zeros(256, dtype=BF16, device="cuda")
    e = torch.empty((0, 256), dtype=BF16, device="cuda")
    assert blk.norm(e, w)["x"].shape == (0, 256)
    R = torch.empty((0, 1024), dtype=BF16, device="cuda")
    out = blk.residual(R, e, torch.empty((0, 4), dtype=BF16, device="cuda"), w, w)
    assert out["R2"].shape == (0, 1024)
    dw = torch.full((256,), 3.0, device="cuda")
    blk.norm_bwd(e, w, torch.empty(0, device="cuda"), e, out={"dw": dw})
    assert bool((dw == 3).all())  # written by no row
    lin = H.Int8Linear(H.LinearConfig(n=32, k=256), 0)
    q = torch.empty((0, 256), dtype=torch.int8, device="cuda")
    wq = torch.zeros((32, 256), dtype=torch.int8, device="cuda")
    assert lin.forward(q, torch.empty(0, device="cuda"), wq, torch.ones(32, device="cuda")).shape == (0, 32)


def test_weight_gradients_of_an_empty_batch_are_zero(H):
    hs = 256
    blk = block(H, 4, hs, BF16)
    w = torch.zeros(hs, dtype=BF16, device="cuda")
    e = {n: torch.empty((0, n), dtype=BF16, device="cuda") for n in (hs, 4 * hs, 4)}
    rr = torch.empty((0, 2), device="cuda")
    for stream in (None, torch.cuda.Stream()):
        held = torch.full((64, hs), 7.0, device="cuda")  # what a new tensor of this size may hold
        del held
        got = [blk.norm_bwd(e[hs], w, rr[:, 0], e[hs], stream=stream)["dw"]]
        out = blk.residual_bwd(e[4 * hs], e[hs], e[4], w, w, rr, e[4 * hs], e[hs], stream=stream)
        got += [out["dw_post"], out["dw_pre"]]
        torch.cuda.synchronize()
        for t in got:
            assert t.shape == (hs,) and not bool(t.any())


def test_zero_rows_and_values_that_are_not_finite(H):
    """A zero row: r = 1/sqrt(eps), q = 0 with scale 0. A row with an infinity
    or a NaN spoils itself and no other row, and its quantized form says so."""
    hs, m = 2560, 6
    for width in (hs, 67, 24576):
        blk, g = block(H, 1, width, BF16), gen(5)
        x, w = randn(g, m, width, dtype=BF16), randn(g, width, dtype=BF16, scale=0.1)
        x[1] = 0
        x[3, width // 2] = float("inf")
        x[4, width - 1] = float("nan")
        out = blk.norm(x, w, out=blk.alloc_norm(m, quantize=True, keep=True))
        good = [0, 2, 5]
        ref = B.norm(x[good], w, EPS)
        B.check(out["x"][good], ref["x"], "x")
        B.check_quantized(out["q"][good], out["q_scale"][good], *ref["x"], "q")
        assert bool((out["x"][1] == 0).all()) and abs(float(out["rrms"][1]) - EPS ** -0.5) < 1e-3
        assert float(out["q_scale"][1]) == 0 and not bool(out["q"][1].any())
        for r in (3, 4):
            assert bool(out["x"][r].isnan().any()) and bool(out["q_scale"][r].isnan()) and not bool(out["q"][r].any())
        lin = H.Int8Linear(H.LinearConfig(n=16, k=width), 0)
        q, s = lin.quantize(x)
        assert bool(s[3].isnan()) and bool(s[4].isnan()) and not bool(q[3:5].any())
        assert float(s[1]) == 0 and not bool(q[1].any())
        wq, ws = lin.quantize(randn(g, 16, width, dtype=BF16))
        o = lin.forward(q, s, wq, ws)
        assert bool(o[3:5].isnan().all()) and bool((o[1] == 0).all()) and bool(o[good].isfinite().all())


def test_large_and_small_magnitudes(H):
    hs, m = 520, 4
    blk = block(H, 1, hs, FP32, eps=0.0)
    g = gen(6)
    w = randn(g, hs, scale=0.1)
    for scale in (1e-15, 1e15):
        x = randn(g, m, hs, scale=scale)
        ref = B.norm(x, w, 0.0)
        out = blk.norm(x, w)
        B.check(out["x"], ref["x"], f"x at {scale}")
    lin = H.Int8Linear(H.LinearConfig(n=1, k=hs, dtype=H.HCGR_FP32), 0)
    for scale in (1e-36, 1e-30, 1e30, 1e37):
        x = randn(g, m, hs, scale=scale)
        q, s = lin.quantize(x)
        B.check_quantized(q, s, x.double(), x.double().abs(), f"q at {scale}")


def test_repeated_calls_are_bitwise_equal(H):
    m, hc, hs = 1500, 4, 2560
    blk, g = block(H, hc, hs, BF16), gen(8)
    i = residual_inputs(g, m, hc, hs, BF16)
    d = {"dR2": randn(g, m, hc * hs, dtype=BF16), "dx": randn(g, m, hs, dtype=BF16)}
    out = blk.residual(**i)
    bwd = blk.residual_bwd(**i, rrms=out["rrms"], **d)
    for _ in range(3):
        again = blk.residual(**i)
        assert all(torch.equal(again[k], out[k]) for k in out)
        b = blk.residual_bwd(**i, rrms=out["rrms"], **d)
        assert all(torch.equal(b[k], bwd[k]) for k in bwd)


def test_rows_are_independent(H):
    """A row's outputs do not depend on the batch it stands in, whichever kernel serves the batch."""
    hc, hs = 4, 2560
    blk, g = block(H, hc, hs, BF16), gen(9)
    i = residual_inputs(g, 3000, hc, hs, BF16)
    out = blk.residual(**i)
    ref = B.residual(**{k: v[:3] if k in ("R", "y", "inj") else v for k, v in i.items()}, hc=hc, eps=EPS, rho=RHO)
    for m in (1, 3):
        few = blk.residual(i["R"][:m], i["y"][:m], i["inj"][:m], i["w_post"], i["w_pre"])
        B.check(few["x"], tuple(t[:m] for t in ref["x"]), "x")
        B.check(few["R2"], tuple(t[:m] for t in ref["R2"]), "R2")
    B.check(out["x"][:3], ref["x"], "x")


# ------------------------------------------------------------------ linear --
LIN = [  # n, k, m
    (1, 1, 1), (3, 5, 2), (16, 16, 1), (17, 63, 16), (15, 64, 17), (64, 65, 64), (100, 1000, 65), (777, 1000, 300),
    (2560, 10240, 1), (10240, 2560, 1), (2560, 10240, 32), (2560, 2560, 5), (320, 10240, 33), (513, 129, 129),
    (1024, 512, 1023), (2500, 640, 513), (4, 131071, 3), (333, 4096, 257), (2560, 320, 2048), (4096, 1040, 1100),
    # few stages of K in many tiles, so that a workgroup's loads run far ahead
    (8200, 40, 8200), (5000, 100, 3000), (4100, 64, 1300), (2600, 130, 1700), (300, 8, 700), (8192, 200, 600),
    # one tile of channels, many of tokens
    (16, 214, 16336), (40, 72, 5000)]


def linear_inputs(g, n, k, m, dt, bias=True, extreme=False):
    def ints(rows):
        pitch = (k + 15) // 16 * 16
        t = torch.randint(-128, 128, (rows, pitch), generator=g, device="cuda", dtype=torch.int16)
        if extreme:
            t = torch.where(t < 0, -128, 127) if rows == m else torch.where(t < 90, -128, 127)
        return t.to(torch.int8)[:, :k]
    return {"q": ints(m), "q_scale": torch.rand(m, generator=g, device="cuda") * 0.1, "w": ints(n),
            "w_scale": torch.rand(n, generator=g, device="cuda") * 0.01,
            "bias": randn(g, n, dtype=dt, scale=3.0) if bias else None}


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("n,k,m", LIN)
def test_linear(H, n, k, m, dt):
    """Integers over all 256 values; the bytes of a row past K hold garbage."""
    say("linear", n, k, m, dt)
    lin = H.Int8Linear(H.LinearConfig(n=n, k=k, dtype=code(H, dt)), 0)
    for bias in (True, False):
        i = linear_inputs(gen(n + k + m), n, k, m, dt, bias)
        if dt is FP16:  # values that fp16 holds
            i["w_scale"] *= 1e-2
        out = lin.forward(**i)
        # the sum is exact; its conversion, the scales' product, the product
        # and the addition round once each: four roundings
        B.check(out, B.linear(**i), "out", 4)


# Shapes of the kernels that LIN does not reach: tiles of outputs that are not
# whole pieces of four, 64 x 64 with a ragged K and N, few tokens with more than
# 4096 channels, streaming stores from 128-token tiles, and 256-token tiles of
# fp32 results that the caches hold.
OTHER_LIN = [(2501, 640, 513), (777, 1000, 2000), (2501, 640, 4000), (8191, 513, 3000), (1023, 513, 1023),
             (777, 1000, 1000), (10240, 2560, 32), (10237, 2561, 20), (5000, 2560, 8), (5003, 2570, 24),
             (2560, 64, 8192), (32772, 640, 129)]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("n,k,m", OTHER_LIN)
def test_linear_of_other_shapes(H, n, k, m, dt):
    test_linear(H, n, k, m, dt)


@pytest.mark.parametrize("n,k,m", [(2500, 640, 513), (2501, 640, 4000), (5000, 100, 3000), (1024, 512, 1023), (10240, 2560, 20)])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_linear_strided_outputs_of_tiles(H, n, k, m, off):
    """Outputs inside a wider tensor, at a start that is and is not a whole
    piece of four: the bits of a dense output, and nothing around it."""
    say("strided tiles", n, k, m, off)
    lin = H.Int8Linear(H.LinearConfig(n=n, k=k), 0)
    i = linear_inputs(gen(n + off), n, k, m, BF16)
    want = lin.forward(**i)
    for pad in (5, 8):
        around = torch.full((m + 1, n + pad), 9.0, dtype=BF16, device="cuda")
        lin.forward(**i, out=around[:m, off:off + n])
        assert torch.equal(around[:m, off:off + n], want)
        assert bool((around[:m, :off] == 9).all()) and bool((around[:m, off + n:] == 9).all())
        assert bool((around[m] == 9).all())


def test_linear_largest_sums(H):
    """All values -128: 131071 products of 2^14 end just below 2^31."""
    k = 131071
    lin = H.Int8Linear(H.LinearConfig(n=20, k=k, dtype=H.HCGR_FP32), 0)
    pitch = (k + 15) // 16 * 16
    for m in (1, 70):
        q = torch.full((m, pitch), -128, dtype=torch.int8, device="cuda")[:, :k]
        w = torch.full((20, pitch), -128, dtype=torch.int8, device="cuda")[:, :k]
        one = torch.ones(m, device="cuda"), torch.ones(20, device="cuda")
        out = lin.forward(q, one[0], w, one[1])
        assert bool((out == float(k) * 2 ** 14).all())  # 131071 * 2^14 is a 32-bit float


@pytest.mark.parametrize("n,k,m", [(100, 300, 5), (64, 300, 1000), (2560, 1000, 600)])
@pytest.mark.parametrize("eq,ew", [(-90, -50), (-50, -90), (-140, 60), (100, -120), (60, -30), (90, 50), (30, 95)])
def test_linear_scales_far_from_one(H, n, k, m, eq, ew):
    """Scales whose product leaves the range of 32 bits (or whose q_scale is
    subnormal) where the results do not; where results would, the tokens are
    zero: bias alone."""
    say("scales", n, k, m, eq, ew)
    lin = H.Int8Linear(H.LinearConfig(n=n, k=k, dtype=H.HCGR_FP32), 0)
    i = linear_inputs(gen(n + m), n, k, m, FP32)
    if eq + ew > 60:
        i["q"].zero_()
    g = gen(eq + 200)
    i["q_scale"] = (1 + torch.rand(m, generator=g, device="cuda")) * 2.0 ** eq
    i["w_scale"] = (1 + torch.rand(n, generator=g, device="cuda")) * 2.0 ** ew
    i["bias"] *= 2.0 ** max(-120, min(60, eq + ew + 10))
    # the sum's conversion, its product with w_scale, and one rounding of the rest
    B.check(lin.forward(**i), B.linear(**i), "out", 2)


@pytest.mark.parametrize("m", [1, 20, 200, 700])
def test_linear_strided(H, m):
    n, k, dt = 200, 300, BF16
    say("linear strided", m)
    lin = H.Int8Linear(H.LinearConfig(n=n, k=k), 0)
    i = linear_inputs(gen(m), n, k, m, dt)
    want = lin.forward(**i)
    wide_q = torch.randint(-128, 127, (m, 1024), device="cuda").to(torch.int8)
    wide_q[:, 32:32 + k] = i["q"]
    wide_w = torch.randint(-128, 127, (n, 512), device="cuda").to(torch.int8)
    wide_w[:, 16:16 + k] = i["w"]
    around = torch.full((m + 1, n + 5), 9.0, dtype=dt, device="cuda")
    lin.forward(wide_q[:, 32:32 + k], i["q_scale"], wide_w[:, 16:16 + k], i["w_scale"], i["bias"],
                out=around[:m, 3:3 + n])
    assert torch.equal(around[:m, 3:3 + n], want)
    assert bool((around[:m, :3] == 9).all()) and bool((around[:m, 3 + n:] == 9).all()) and bool((around[m] == 9).all())


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("k,m", [(1, 3), (40, 5), (67, 9), (2560, 1), (10240, 33), (20000, 4), (131071, 2)])
def test_quantize(H, k, m, dt):
    say("quantize", k, m, dt)
    lin = H.Int8Linear(H.LinearConfig(n=8, k=k, dtype=code(H, dt)), 0)
    x = randn(gen(k), m, k, dtype=dt, scale=5.0)
    q, s = lin.quantize(x)
    B.check_quantized(q, s, x.double(), x.double().abs(), "q", 4)


def test_quantize_ties_go_to_even(H):
    """scale = 1 exactly: x.5 rounds to the even neighbour."""
    lin = H.Int8Linear(H.LinearConfig(n=8, k=8, dtype=H.HCGR_FP32), 0)
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 126.5]], device="cuda")
    q, s = lin.quantize(x)
    assert float(s) == 1.0 and q.tolist() == [[127, 0, 2, 2, 0, -2, -126, 126]]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("k", [256, 2000, 20480])
def test_quantize_ties_at_any_scale(H, k, dt):
    """Every scale s whose s*127 and (i + 1/2)*s the type holds: the quotients
    are exact ties, whatever 1/s is."""
    say("ties", k, dt)
    bits = {BF16: 8, FP16: 11, FP32: 24}[dt]
    steps = [s for s in range(1, 1 << min(bits - 7, 12)) if s * 127 < 1 << bits] + [0.25, 0.5]
    half = torch.arange(-126.5, 127.5, 1.0)
    x = torch.zeros(len(steps), k)
    x[:, 0] = 127 * torch.tensor(steps)
    x[:, 1:255] = half[None, :] * torch.tensor(steps)[:, None]
    held = x.to(dt).float() == x  # the others (many bits) are left out
    x = torch.where(held, x, 0.0)
    assert bool(held[:, 0].all()) and int((x[:, 1:] != 0).sum()) >= 60 * len(steps)
    lin = H.Int8Linear(H.LinearConfig(n=8, k=k, dtype=code(H, dt)), 0)
    q, s = lin.quantize(x.to(dt).cuda())
    assert torch.equal(s.cpu(), torch.tensor(steps, dtype=FP32))
    want = torch.round(x.double() / torch.tensor(steps, dtype=torch.float64)[:, None])  # half to even
    assert torch.equal(q.cpu().double(), want)


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("k,m", [(2560, 300), (67, 3000), (20480, 40)])
def test_quantize_is_the_rounded_quotient(H, k, m, dt):
    """q is v/q_scale in 32 bits, rounded: the remainder step leaves the quotient
    within 2^-44 of itself, so that only a quotient that close to the middle of
    two 32-bit values next to a half could differ (one in some 10^8)."""
    lin = H.Int8Linear(H.LinearConfig(n=8, k=k, dtype=code(H, dt)), 0)
    x = randn(gen(k + m), m, k, dtype=dt, scale=3.0)
    q, s = lin.quantize(x)
    x, s = x.float().cpu(), s.cpu()
    assert torch.equal(s, x.abs().amax(1) / 127)
    assert torch.equal(q.cpu().float(), torch.round(x / s[:, None]))


# ------------------------------------------------------- refusals in Python --
def test_wrong_tensors_are_refused(H):
    blk = block(H, 2, 64, BF16)
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    w = torch.zeros(64, dtype=BF16, device="cuda")
    bad = [lambda: blk.norm(x.float(), w), lambda: blk.norm(x, w.float()), lambda: blk.norm(x[:, :32], w),
           lambda: blk.norm(x.cpu(), w), lambda: blk.norm(x.t().contiguous().t(), w), lambda: blk.norm(x, w[:63]),
           lambda: blk.norm(x, w, out={"x": torch.zeros((3, 64), dtype=BF16, device="cuda")}),
           lambda: blk.residual(x, x, None, w, w), lambda: blk.norm_bwd(x, w, torch.zeros(3, device="cuda"), x)]
    lin = H.Int8Linear(H.LinearConfig(n=8, k=40), 0)
    q, s = torch.zeros((4, 40), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    wq = torch.zeros((8, 48), dtype=torch.int8, device="cuda")[:, :40]
    ws = torch.zeros(8, device="cuda")
    bad += [lambda: lin.forward(q, s, wq, ws),                 # rows of 40 bytes have no whole last piece
            lambda: lin.forward(q[:1, :39], s[:1], wq, ws), lambda: lin.forward(wq[:4], s, wq, ws.double()),
            lambda: lin.quantize(x[:, :40].float()), lambda: lin.forward(wq[:4], s[:3], wq, ws)]
    for k, f in enumerate(bad):
        with pytest.raises((ValueError, H.HcgrError)):
            f()
            pytest.fail(f"call {k} was accepted")
    with pytest.raises(H.HcgrError) as e:  # overlapping rows
        blk.norm(x[0].expand(4, 64), w)
    assert e.value.status == H.HCGR_ERR_INVALID_ARGUMENT


def test_quantize_that_cannot_be_answered_is_refused(H):
    blk, g = block(H, 2, 64, BF16), gen(50)
    i = residual_inputs(g, 4, 2, 64, BF16)
    x, w = i["y"], i["w_pre"]
    plain, both = blk.alloc_norm(4), blk.alloc_norm(4, quantize=True, keep=True)
    with pytest.raises(ValueError, match="quantize"):
        blk.norm(x, w, quantize=True, out=plain)
    with pytest.raises(ValueError, match="quantize"):
        blk.residual(**i, quantize=True, out=blk.alloc_residual(4))
    with pytest.raises(ValueError, match="quantize"):
        blk.residual(i["R"], x, i["inj"], i["w_post"], None, quantize=True)
    with pytest.raises(ValueError, match="quantize"):
        blk.residual(i["R"], x, i["inj"], i["w_post"], None, quantize=True, out=blk.alloc_residual(4, norm=False))
    want = blk.norm(x, w, quantize=True)
    for out in (blk.norm(x, w, quantize=True, out=both), blk.norm(x, w, out=both)):
        assert torch.equal(out["q"], want["q"]) and torch.equal(out["x"], blk.norm(x, w)["x"])


# --------------------------------------------------------------- as a layer --
class Layer:
    """mix -> norm (quantized) -> linear -> SiLU -> quantize -> linear ->
    residual, on HCGR's own shapes, in a program's way."""

    def __init__(self, H, hc=4, hs=1280, wide=2560, seed=0):
        import synth
        self.shape = synth.Shape(hc=hc, hs=hs, r=64)
        self.hw = synth.make_weights(self.shape, seed=seed, device="cuda")
        self.op = H.HCGR(H.Config(hc=hc, hs=hs, r=64), 0)
        self.one, self.blk = block(H, 1, hs, BF16), block(H, hc, hs, BF16)
        self.up = H.Int8Linear(H.LinearConfig(n=wide, k=hs), 0)
        self.down = H.Int8Linear(H.LinearConfig(n=hs, k=wide), 0)
        g = gen(seed)
        self.w = [randn(g, hs, dtype=BF16, scale=0.1) for _ in range(3)]
        self.w_up = self.up.quantize(randn(g, wide, hs, dtype=BF16, scale=hs ** -0.5))
        self.w_down = self.down.quantize(randn(g, hs, wide, dtype=BF16, scale=wide ** -0.5))

    def __call__(self, R, inj, workspace=None):
        m = self.op.mix(R, *(self.hw[k] for k in ("wnorm", "wd", "wi", "wu")), workspace=workspace)
        n = self.one.norm(m["x"], self.w[0], quantize=True)
        a = torch.nn.functional.silu(self.up.forward(n["q"], n["q_scale"], *self.w_up))
        y = self.down.forward(*self.down.quantize(a), *self.w_down)
        out = self.blk.residual(R, y, inj, self.w[1], self.w[2])
        return {"mixed": m["x"], "n": n, "a": a, "y": y, **out}


def layer_inputs(layer, m, seed):
    g = gen(seed)
    s = layer.shape
    return randn(g, m, s.hc * s.hs, dtype=BF16), randn(g, m, s.hc, dtype=BF16)


@pytest.mark.parametrize("m", [1, 33, 300])
def test_a_layer_of_the_operators(H, m):
    """Each step of the run against the 64-bit form of that step on what the
    step before it gave."""
    layer = Layer(H)
    R, inj = layer_inputs(layer, m, m)
    o = layer(R, inj)
    ref = B.norm(o["mixed"], layer.w[0], EPS)
    B.check_quantized(o["n"]["q"], o["n"]["q_scale"], *ref["x"], "q")
    up = B.linear(o["n"]["q"], o["n"]["q_scale"], *layer.w_up, None)
    got = layer.up.forward(o["n"]["q"], o["n"]["q_scale"], *layer.w_up)
    B.check(got, up, "up", 4)
    q, s = layer.down.quantize(o["a"])
    B.check(o["y"], B.linear(q, s, *layer.w_down, None), "down", 4)
    ref = B.residual(R, o["y"], inj, layer.w[1], layer.w[2], hc=layer.shape.hc, eps=EPS, rho=RHO)
    check_residual(o, ref, True, True)


def test_layer_in_a_graph(H):
    """Captured once, replayed with new inputs between eager calls: each replay
    equals the eager result. Two graphs of one set of handles are replayed on
    two streams (HCGR's own calls with a workspace for each graph)."""
    layer, m = Layer(H), 20
    bufs, graphs, outs, spaces = [], [], [], []
    for k in range(2):
        R, inj = layer_inputs(layer, m, k)
        layer(R, inj)
        spaces.append(H.new_workspace(H.hcgr_workspace_size(layer.op.handle, m)))
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(layer(R, inj, spaces[k]))
        bufs.append((R, inj))
        graphs.append(gr)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for k in range(2):
            R, inj = layer_inputs(layer, m, 10 * rep + k)
            bufs[k][0].copy_(R)
            bufs[k][1].copy_(inj)
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            want = layer(*bufs[k])
            torch.cuda.synchronize()
            for name in ("y", "R2", "x", "rrms"):
                assert torch.equal(outs[k][name], want[name]), (rep, k, name)


def test_backward_in_a_graph(H):
    m, hc, hs = 600, 4, 1280
    blk, g = block(H, hc, hs, BF16), gen(11)
    i = residual_inputs(g, m, hc, hs, BF16)
    d = {"dR2": randn(g, m, hc * hs, dtype=BF16), "dx": randn(g, m, hs, dtype=BF16)}
    rrms = blk.residual(**i)["rrms"].clone()
    blk.residual_bwd(**i, rrms=rrms, **d)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        f = blk.residual(**i)
        b = blk.residual_bwd(**i, rrms=f["rrms"], **d)
    for rep in range(4):
        i["y"].copy_(randn(g, m, hs, dtype=BF16))
        d["dx"].copy_(randn(g, m, hs, dtype=BF16))
        gr.replay()
        torch.cuda.synchronize()
        f2 = blk.residual(**i)
        b2 = blk.residual_bwd(**i, rrms=f2["rrms"], **d)
        torch.cuda.synchronize()
        assert all(torch.equal(f[k], f2[k]) for k in f2) and all(torch.equal(b[k], b2[k]) for k in b2), rep


def test_other_streams(H):
    """Calls given another stream than torch's current one, outputs and
    workspaces allocated by the call."""
    m, hc, hs = 400, 2, 1000
    blk, g = block(H, hc, hs, BF16), gen(12)
    i = residual_inputs(g, m, hc, hs, BF16)
    d = {"dR2": randn(g, m, hc * hs, dtype=BF16), "dx": randn(g, m, hs, dtype=BF16)}
    f = blk.residual(**i)
    b = blk.residual_bwd(**i, rrms=f["rrms"], **d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        f2 = blk.residual(**i, stream=stream)
        b2 = blk.residual_bwd(**i, rrms=f2["rrms"], **d, stream=stream)
        s.synchronize()
        assert all(torch.equal(f[k], f2[k]) for k in f) and all(torch.equal(b[k], b2[k]) for k in b)


# ------------------------------------------------- far offsets, many callers --
def test_offsets_past_32_bits(H):
    """Tensors of more than 2^32 bytes: the first and last rows, and rows
    around the 2^31 and 2^32 byte marks."""
    m, hc, hs = 110000, 8, 2560
    say("far residual")
    blk = block(H, hc, hs, BF16)
    g = gen(20)
    i = residual_inputs(g, 1, hc, hs, BF16)
    i["y"], i["inj"] = randn(g, m, hs, dtype=BF16), randn(g, m, hc, dtype=BF16)
    i["R"] = torch.empty((m, hc * hs), dtype=BF16, device="cuda")
    for a in range(0, m, 10000):
        i["R"][a:a + 10000] = randn(g, min(10000, m - a), hc * hs, dtype=BF16)
    assert i["R"].numel() * 2 > 2 ** 32
    marks = [0, 1, 52428, 52429, 104857, 104858, m - 1]
    out = blk.residual(**i)
    few = {k: (v[marks] if k in ("R", "y", "inj") else v) for k, v in i.items()}
    ref = B.residual(**few, hc=hc, eps=EPS, rho=RHO)
    check_residual({k: v[marks] for k, v in out.items()}, ref, True, True)
    dx = randn(g, m, hs, dtype=BF16)
    got = blk.residual_bwd(**i, rrms=out["rrms"], dR2=i["R"], dx=dx)
    want = B.residual_bwd(**few, rrms=out["rrms"][marks], dR2=i["R"][marks], dx=dx[marks], hc=hc, rho=RHO)
    for k in ("dR", "dy", "dinj"):
        B.check(got[k][marks], want[k], k)


@pytest.mark.parametrize("n,k,m", [(8192, 64, 300000), (16, 32, 1100000), (1048576, 4112, 3), (40000, 48, 60000)])
def test_linear_offsets_past_32_bits(H, n, k, m):
    """Outputs or weights of more than 2^32 bytes, and more than 2^20 tokens."""
    say("far linear", n, k, m)
    lin = H.Int8Linear(H.LinearConfig(n=n, k=k), 0)
    i = linear_inputs(gen(21), n, k, m, BF16)
    out = lin.forward(**i)
    rows = sorted({0, 1, m // 2, m - 2, m - 1} & set(range(m)) | ({1 << 20, (1 << 20) - 1} if m > 1 << 20 else set()))
    cols = sorted({0, 1, n // 2, n - 2, n - 1})
    part = {"q": i["q"][rows], "q_scale": i["q_scale"][rows], "w": i["w"][cols], "w_scale": i["w_scale"][cols],
            "bias": i["bias"][cols]}
    B.check(out[rows][:, cols], B.linear(**part), "out", 4)


def test_two_threads_on_one_handle(H):
    """Handles are read-only: two threads call them at once, each on a stream of its own."""
    import threading
    m, hc, hs = 900, 2, 1000
    blk, lin = block(H, hc, hs, BF16), H.Int8Linear(H.LinearConfig(n=300, k=hs), 0)
    sets, want, got = [], [], [None, None]
    for t in range(2):
        g = gen(30 + t)
        i = residual_inputs(g, m, hc, hs, BF16)
        d = {"dR2": randn(g, m, hc * hs, dtype=BF16), "dx": randn(g, m, hs, dtype=BF16)}
        w = lin.quantize(randn(g, 300, hs, dtype=BF16))
        sets.append((i, d, w))

    def run(t, reps):
        i, d, w = sets[t]
        for _ in range(reps):
            f = blk.residual(**i, quantize=True)
            b = blk.residual_bwd(**i, rrms=f["rrms"], **d)
            o = lin.forward(f["q"], f["q_scale"], *w)
        return {**f, **b, "o": o}

    want = [run(t, 1) for t in range(2)]
    torch.cuda.synchronize()

    def worker(t):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got[t] = run(t, 20)
        s.synchronize()

    threads = [threading.Thread(target=worker, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for t in range(2):
        assert all(torch.equal(got[t][k], want[t][k]) for k in want[t]), t


def test_outputs_for_another_stream_are_that_stream_s_memory(H):
    """A block that torch's current stream has freed but still writes is not
    handed to a call on another stream."""
    m, hs = 4096, 2560
    blk, g = block(H, 1, hs, BF16), gen(41)
    x, w = randn(g, m, hs, dtype=BF16), randn(g, hs, dtype=BF16, scale=0.1)
    want = blk.norm(x, w)["x"].clone()
    big = torch.randn(8192, 8192, device="cuda")
    s = torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        held = torch.empty((m, hs), dtype=BF16, device="cuda")
        torch.mm(big, big)           # keeps the current stream busy
        held.fill_(7.0)              # pending when the block is freed
        del held
        out = blk.norm(x, w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out["x"], want)


def test_more_rows_than_one_launch_takes(H):
    """Past 2^28 rows of one value, four to a workgroup of 64 x 4 threads, a
    launch would pass 2^32 threads: the call takes several. Every row is
    written, and the rows around each launch's ends are right."""
    m = (1 << 28) + 37
    say("many rows", m)
    blk, g = block(H, 1, 1, BF16), gen(22)
    x, w = randn(g, m, 1, dtype=BF16, scale=3.0), randn(g, 1, dtype=BF16, scale=0.2)
    out = {"x": torch.full((m, 1), float("nan"), dtype=BF16, device="cuda"),
           "rrms": torch.full((m,), float("nan"), device="cuda")}
    blk.norm(x, w, out=out)
    assert bool(out["x"].isfinite().all()) and bool(out["rrms"].isfinite().all())
    rows = torch.tensor([r + d for r in (0, 1 << 27, 1 << 28, m) for d in range(-6, 6) if 0 <= r + d < m], device="cuda")
    ref = B.norm(x[rows], w, EPS)
    B.check(out["x"][rows], ref["x"], "x")
    B.check(out["rrms"][rows], ref["rrms"], "rrms")


def test_combine_of_more_tokens_than_one_launch_takes(H):
    """Past 2^22 tokens of four streams a launch of the op's combine would pass
    2^32 threads."""
    m, hc, hs = (1 << 22) + 37, 4, 128
    say("many tokens", m)
    op, g = H.HCGR(H.Config(hc=hc, hs=hs, r=32), 0), gen(23)
    R = torch.empty((m, hc * hs), dtype=BF16, device="cuda")
    for a in range(0, m, 1 << 20):
        R[a:a + (1 << 20)] = randn(g, min(1 << 20, m - a), hc * hs, dtype=BF16)
    y, inj = randn(g, m, hs, dtype=BF16), randn(g, m, hc, dtype=BF16)
    R2 = torch.full_like(R, float("nan"))
    op.combine(R, y, inj, R2=R2)
    assert not bool(R2.isnan().any())
    rows = torch.tensor([r + d for r in (0, 1 << 21, 1 << 22, m) for d in range(-9, 9) if 0 <= r + d < m], device="cuda")
    ref = B.residual(R[rows], y[rows], inj[rows], None, None, hc=hc, eps=EPS, rho=1.0)
    B.check(R2[rows], ref["R2"], "R2")
