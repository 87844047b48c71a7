"""The error contract of the block operators on the CPU: hcgr_validate_block_*
and hcgr_validate_linear_* run the checks of their entry points on plain
addresses, without a GPU or a launch."""
import ctypes
import os

import pytest

import skinny_gemm_hcgr_amd as H

OK, INVALID, UNSUPPORTED, ALIASING, SMALL = (H.HCGR_OK, H.HCGR_ERR_INVALID_ARGUMENT, H.HCGR_ERR_UNSUPPORTED,
                                             H.HCGR_ERR_ALIASING, H.HCGR_ERR_WORKSPACE_TOO_SMALL)
BYTES = {H.HCGR_BF16: 2, H.HCGR_FP16: 2, H.HCGR_FP32: 4}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(H.LIB_PATH):
        from skinny_gemm_hcgr_amd import build
        build.build()
    return H.load_library()


def layout(sizes):
    """Disjoint 256-byte aligned addresses, never dereferenced."""
    a, out = 1 << 32, {}
    for k, n in sizes.items():
        out[k] = a
        a += (n + 4096 + 255) // 256 * 256
    return out


class Norm:
    names = ("x", "ld_x", "w", "M", "xn", "q", "ld_q", "q_scale", "rrms")
    validate = staticmethod(lambda *a: H.hcgr_validate_block_norm(*a))
    required = ("x", "w", "q_scale", "q")
    optional = ("rrms", "xn")

    def __init__(self, M=5, hs=40, dtype=H.HCGR_BF16):
        b, ldq = BYTES[dtype], (hs + 15) // 16 * 16
        self.cfg = H.BlockConfig(hc=1, hs=hs, dtype=dtype)
        self.sizes = {"x": M * hs * b, "w": hs * b, "xn": M * hs * b, "q": M * ldq, "q_scale": M * 4, "rrms": M * 4}
        self.args = {**layout(self.sizes), "ld_x": hs, "ld_q": ldq, "M": M}
        self.outputs = ("xn", "q", "q_scale", "rrms")

    def call(self, **over):
        a = {**self.args, **over}
        return type(self).validate(a.pop("cfg", self.cfg), *(a[n] for n in self.names))


class NormBwd(Norm):
    names = ("x", "ld_x", "w", "rrms", "dxn", "M", "dx", "dw", "ws", "ws_bytes")
    validate = staticmethod(lambda *a: H.hcgr_validate_block_norm_bwd(*a))
    required = ("x", "w", "rrms", "dxn", "ws")
    optional = ("dx", "dw")

    def __init__(self, M=5, hs=40, dtype=H.HCGR_BF16):
        b = BYTES[dtype]
        self.cfg = H.BlockConfig(hc=1, hs=hs, dtype=dtype)
        n = H.hcgr_block_workspace_size_for(self.cfg, M)
        self.sizes = {"x": M * hs * b, "w": hs * b, "rrms": M * 4, "dxn": M * hs * b, "dx": M * hs * b, "dw": hs * 4,
                      "ws": n}
        self.args = {**layout(self.sizes), "ld_x": hs, "M": M, "ws_bytes": n}
        self.outputs = ("dx", "dw", "ws")


class Residual(Norm):
    names = ("R", "y", "ld_y", "inj", "ld_inj", "w_post", "w_pre", "M", "R2", "x", "q", "ld_q", "q_scale", "rrms")
    validate = staticmethod(lambda *a: H.hcgr_validate_block_residual(*a))
    required = ("R", "y", "R2", "w_pre", "q_scale", "q")
    optional = ("inj", "w_post", "x", "rrms")

    def __init__(self, M=5, hs=40, dtype=H.HCGR_BF16, hc=4):
        b, ldq = BYTES[dtype], (hs + 15) // 16 * 16
        self.cfg = H.BlockConfig(hc=hc, hs=hs, dtype=dtype)
        self.sizes = {"R": M * hc * hs * b, "y": M * hs * b, "inj": M * hc * b, "w_post": hs * b, "w_pre": hs * b,
                      "R2": M * hc * hs * b, "x": M * hs * b, "q": M * ldq, "q_scale": M * 4, "rrms": M * 8}
        self.args = {**layout(self.sizes), "ld_y": hs, "ld_inj": hc, "ld_q": ldq, "M": M}
        self.outputs = ("R2", "x", "q", "q_scale", "rrms")


class ResidualBwd(Norm):
    names = ("R", "y", "ld_y", "inj", "ld_inj", "w_post", "w_pre", "rrms", "dR2", "dx", "M", "dR", "dy", "dinj",
             "ld_dinj", "dw_post", "dw_pre", "ws", "ws_bytes")
    validate = staticmethod(lambda *a: H.hcgr_validate_block_residual_bwd(*a))
    required = ("R", "y", "rrms", "dx", "dR", "dy", "inj", "w_post", "w_pre", "dinj", "dw_post", "dw_pre", "ws")
    optional = ("dR2",)

    def __init__(self, M=5, hs=40, dtype=H.HCGR_BF16, hc=4):
        b = BYTES[dtype]
        self.cfg = H.BlockConfig(hc=hc, hs=hs, dtype=dtype)
        n = H.hcgr_block_workspace_size_for(self.cfg, M)
        row, k = hs * b, hc * hs * b
        self.sizes = {"R": M * k, "y": M * row, "inj": M * hc * b, "w_post": row, "w_pre": row, "rrms": M * 8,
                      "dR2": M * k, "dx": M * row, "dR": M * k, "dy": M * row, "dinj": M * hc * b, "dw_post": hs * 4,
                      "dw_pre": hs * 4, "ws": n}
        self.args = {**layout(self.sizes), "ld_y": hs, "ld_inj": hc, "ld_dinj": hc, "M": M, "ws_bytes": n}
        self.outputs = ("dR", "dy", "dinj", "dw_post", "dw_pre", "ws")


class Quantize(Norm):
    names = ("x", "ld_x", "M", "q", "ld_q", "q_scale")
    validate = staticmethod(lambda *a: H.hcgr_validate_linear_quantize(*a))
    required = ("x", "q", "q_scale")
    optional = ()

    def __init__(self, M=5, hs=40, dtype=H.HCGR_BF16):
        ldq = (hs + 15) // 16 * 16
        self.cfg = H.LinearConfig(n=24, k=hs, dtype=dtype)
        self.sizes = {"x": M * hs * BYTES[dtype], "q": M * ldq, "q_scale": M * 4}
        self.args = {**layout(self.sizes), "ld_x": hs, "ld_q": ldq, "M": M}
        self.outputs = ("q", "q_scale")


class Linear(Norm):
    names = ("q", "ld_q", "q_scale", "w", "ld_w", "w_scale", "bias", "M", "out", "ld_out")
    validate = staticmethod(lambda *a: H.hcgr_validate_linear_forward(*a))
    required = ("q", "q_scale", "w", "w_scale", "out")
    optional = ("bias",)

    def __init__(self, M=5, hs=40, dtype=H.HCGR_BF16, n=24):
        b, ld = BYTES[dtype], (hs + 15) // 16 * 16
        self.cfg = H.LinearConfig(n=n, k=hs, dtype=dtype)
        self.sizes = {"q": M * ld, "q_scale": M * 4, "w": n * ld, "w_scale": n * 4, "bias": n * b, "out": M * n * b}
        self.args = {**layout(self.sizes), "ld_q": ld, "ld_w": ld, "ld_out": n, "M": M}
        self.outputs = ("out",)


CALLS = [Norm, NormBwd, Residual, ResidualBwd, Quantize, Linear]
each = pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)


@each
@pytest.mark.parametrize("dtype", list(BYTES))
@pytest.mark.parametrize("M,hs", [(1, 1), (3, 67), (5, 2560), (70000, 65536)])
def test_valid_calls_pass(call, dtype, M, hs):
    assert call(M, hs, dtype).call() == OK, H.last_error()


@each
def test_m_zero_is_a_no_op_even_with_null_pointers(call):
    c = call()
    assert c.call(M=0, **{n: None for n in c.sizes}) == OK
    assert c.call(M=-1) == INVALID
    assert c.call(M=(1 << 31) + 1) == UNSUPPORTED


@each
def test_null_and_misaligned_pointers(call):
    c = call()
    for n in c.required:
        assert c.call(**{n: 0}) == INVALID, n
    for n in c.optional:
        assert c.call(**{n: 0}) == OK, n
    for n in c.sizes:
        assert c.call(**{n: c.args[n] + 1}) == INVALID, n
        if n in ("q", "w", "ws") and not (n == "w" and call in (Norm, NormBwd)):
            assert c.call(**{n: c.args[n] + 8}) == INVALID, n
        elif n in ("q_scale", "rrms", "dw", "dw_post", "dw_pre", "w_scale"):
            assert c.call(**{n: c.args[n] + 2}) == INVALID, n


@each
def test_outputs_that_overlap(call):
    c = call(M=70, hs=64)
    for o in c.outputs:
        for n in c.sizes:
            if n != o:
                assert c.call(**{o: c.args[n]}) == ALIASING, (o, n)
        assert {"ws": "workspace"}.get(o, o) in H.last_error()


@each
def test_leading_dimensions(call):
    c = call()
    for n in c.names:
        if n.startswith("ld_"):
            assert c.call(**{n: c.args[n] - 16}) == INVALID, n
            assert c.call(**{n: c.args[n] + 16}) == OK, n
            assert c.call(**{n: (1 << 31) + 16}) == UNSUPPORTED, n
        if n in ("ld_q", "ld_w"):
            assert c.call(**{n: c.args[n] + 8}) == INVALID, n
    if call is Linear:
        c = Linear(M=1, n=1)  # one row each: its pitch does not widen the matrix
        for n in ("ld_q", "ld_w"):
            assert c.call(**{n: H.HCGR_LINEAR_MAX_LD}) == OK
            assert c.call(**{n: H.HCGR_LINEAR_MAX_LD + 16}) == UNSUPPORTED


@pytest.mark.parametrize("call", [NormBwd, ResidualBwd], ids=lambda c: c.__name__)
def test_workspace_too_small(call):
    c = call(M=1000, hs=200)
    assert c.call(ws_bytes=c.args["ws_bytes"] - 1) == SMALL
    cfg = c.cfg
    sizes = [H.hcgr_block_workspace_size_for(cfg, m) for m in (0, 1, 2, 3, 511, 512, 513, 100000)]
    assert sizes[0] == 0 and sizes == sorted(sizes)


def test_outputs_that_belong_together():
    c = Norm()
    assert c.call(xn=0, q=0, q_scale=0) == INVALID      # nothing to write
    assert c.call(q=0, q_scale=0) == OK
    b = NormBwd()
    assert b.call(dx=0, dw=0) == INVALID
    r = Residual()
    assert r.call(x=0, q=0, q_scale=0) == INVALID       # w_pre without x or q
    assert r.call(w_pre=0) == INVALID                   # x and q without w_pre
    assert r.call(w_pre=0, x=0, q=0, q_scale=0) == OK
    g = ResidualBwd()
    assert g.call(dR2=0, dx=0, w_pre=0, dw_pre=0) == INVALID
    assert g.call(dx=0, w_pre=0, dw_pre=0) == OK
    assert g.call(inj=0, dinj=0) == OK
    assert g.call(w_post=0, dw_post=0) == OK
    assert g.call(w_post=0, dw_post=0, w_pre=0, dw_pre=0, dx=0, rrms=0) == OK


@pytest.mark.parametrize("over,status", [
    ({"hc": 3}, UNSUPPORTED), ({"hc": 0}, INVALID), ({"hs": 0}, INVALID), ({"hs": 65537}, UNSUPPORTED),
    ({"dtype": 3}, INVALID), ({"dtype": -1}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"res_scale": float("inf")}, INVALID)])
def test_block_configurations(over, status):
    cfg = H.BlockConfig(**{"hc": 1, "hs": 40, **over})
    assert Norm().call(cfg=cfg) == status
    with pytest.raises(H.HcgrError) as e:
        H.hcgr_block_workspace_size_for(cfg, 4)
    assert e.value.status == status
    with pytest.raises(H.HcgrError) as e:
        H.hcgr_block_create(cfg, 0)
    assert e.value.status == status


@pytest.mark.parametrize("over,status", [
    ({"n": 0}, INVALID), ({"k": 0}, INVALID), ({"k": H.HCGR_LINEAR_MAX_K + 1}, UNSUPPORTED),
    ({"n": H.HCGR_LINEAR_MAX_N + 1}, UNSUPPORTED), ({"dtype": 7}, INVALID)])
def test_linear_configurations(over, status):
    cfg = H.LinearConfig(**{"n": 24, "k": 40, **over})
    assert Linear().call(cfg=cfg) == status
    with pytest.raises(H.HcgrError) as e:
        H.hcgr_linear_create(cfg, 0)
    assert e.value.status == status


def test_null_config_and_handle(lib):
    n = ctypes.c_size_t()
    assert lib.hcgr_block_create(None, 0, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.hcgr_linear_create(None, 0, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert lib.hcgr_block_create(ctypes.byref(H.BlockConfig().c()), 0, None) == INVALID
    assert lib.hcgr_block_workspace_size(None, 4, ctypes.byref(n)) == INVALID
    assert lib.hcgr_block_workspace_size_for(ctypes.byref(H.BlockConfig().c()), 4, None) == INVALID
    lib.hcgr_block_destroy(None)
    lib.hcgr_linear_destroy(None)
    c = Linear()
    assert lib.hcgr_linear_forward(None, *(c.args[n] for n in c.names), None) == INVALID
    assert lib.hcgr_block_norm(None, *(Norm().args[n] for n in Norm.names), None) == INVALID


def test_bytes_past_k_belong_to_the_row():
    """The last row of q and w is read up to a whole 16-byte piece: an output
    that starts inside that piece overlaps it."""
    c = Linear(M=3, hs=40)
    end = c.args["q"] + 2 * 48 + 40
    assert c.call(out=end) == ALIASING
    assert c.call(out=end + 8) == OK
