"""The launches of the block operators on the CPU: what each call sends to the
device, recorded by a stand-in for the HIP runtime."""
import os
import re

import pytest

import skinny_gemm_hcgr_amd as H
from launch_record import BLOCK, GRID, Recorder

BYTES = {H.HCGR_BF16: 2, H.HCGR_FP16: 2, H.HCGR_FP32: 4}


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    if not os.path.exists(H.LIB_PATH):
        from skinny_gemm_hcgr_amd import build
        build.build()
    r = Recorder(tmp_path_factory.mktemp("runtime"))
    yield r
    r.close()


def places(*sizes):
    """Disjoint addresses, never dereferenced; 256-byte aligned."""
    at, out = 1 << 32, []
    for n in sizes:
        out.append(at)
        at += (n + 255) // 256 * 256
    return out


def norm(rec, M, hs, dtype=H.HCGR_BF16, shift=0, **q):
    b, ldq = BYTES[dtype], (hs + 15) // 16 * 16
    x, w, xn, qq, qs, rr = places(M * hs * b + 64, hs * b, M * hs * b, M * ldq, 4 * M, 4 * M)
    return rec.ask(config="BlockConfig", values={"hc": 1, "hs": hs, "dtype": dtype}, call="hcgr_block_norm",
                   args=[x + shift, hs, w, M, xn, qq, ldq, qs, rr], **q)


def residual(rec, M, hs, hc, dtype=H.HCGR_BF16, **q):
    b = BYTES[dtype]
    R, y, inj, w, R2, x, rr = places(M * hc * hs * b, M * hs * b, M * hc * b, hs * b, M * hc * hs * b, M * hs * b, 8 * M)
    return rec.ask(config="BlockConfig", values={"hc": hc, "hs": hs, "dtype": dtype}, call="hcgr_block_residual",
                   args=[R, y, hs, inj, hc, w, w, M, R2, x, None, 0, None, rr], **q)


def quantize(rec, M, k, dtype=H.HCGR_BF16, **q):
    ldq = (k + 15) // 16 * 16
    x, qq, qs = places(M * k * BYTES[dtype], M * ldq, 4 * M)
    return rec.ask(config="LinearConfig", values={"n": 8, "k": k, "dtype": dtype}, call="hcgr_linear_quantize",
                   args=[x, k, M, qq, ldq, qs], **q)


def backward(rec, M, hs, hc, dtype=H.HCGR_BF16, **q):
    b = BYTES[dtype]
    n = H.hcgr_block_workspace_size_for(H.BlockConfig(hc=hc, hs=hs, dtype=dtype), M)
    row, k = hs * b, hc * hs * b
    R, y, inj, w, rr, dR2, dx, dR, dy, dinj, dw, dw2, ws = places(M * k, M * row, M * hc * b, row, 8 * M, M * k, M * row,
                                                                  M * k, M * row, M * hc * b, hs * 4, hs * 4, n)
    return rec.ask(config="BlockConfig", values={"hc": hc, "hs": hs, "dtype": dtype}, call="hcgr_block_residual_bwd",
                   args=[R, y, hs, inj, hc, w, w, rr, dR2, dx, M, dR, dy, dinj, hc, dw, dw2, ws, n], **q)


def norm_backward(rec, M, hs, dtype=H.HCGR_BF16, **q):
    b = BYTES[dtype]
    ws_bytes = H.hcgr_block_workspace_size_for(H.BlockConfig(hc=1, hs=hs, dtype=dtype), M)
    x, w, rr, d, dx, dw, ws = places(M * hs * b, hs * b, 4 * M, M * hs * b, M * hs * b, 4 * hs, ws_bytes)
    return rec.ask(config="BlockConfig", values={"hc": 1, "hs": hs, "dtype": dtype}, call="hcgr_block_norm_bwd",
                   args=[x, hs, w, rr, d, M, dx, dw, ws, ws_bytes], **q)


def linear(rec, M, n, k, dtype=H.HCGR_BF16, ld_out=None, shift=0, **q):
    b, ld, ld_out = BYTES[dtype], (k + 15) // 16 * 16, ld_out or n
    x, qs, w, ws, bias, out = places(M * ld, 4 * M, n * ld, 4 * n, n * b, M * ld_out * b + 64)
    return rec.ask(config="LinearConfig", values={"n": n, "k": k, "dtype": dtype}, call="hcgr_linear_forward",
                   args=[x, ld, qs, w, ld, ws, bias, M, out + shift, ld_out], **q)


def check_sizes(answer):
    """Every launch within what HIP supports: fewer than 2^32 threads in a
    dimension (gridDim x blockDim), 1024 in a workgroup, 160 KB of LDS."""
    assert answer["status"] == H.HCGR_OK, answer["error"]
    assert answer["launches"]
    for la in answer["launches"]:
        for g, b in zip(GRID, BLOCK):
            assert 1 <= la[g] < 1 << 31 and la[g] * la[b] < 1 << 32, la
        assert la["bx"] * la["by"] * la["bz"] <= 1024 and la["lds"] <= 160 * 1024, la
    return answer["launches"]


def rows_of(launches):
    return sum(la["gx"] * la["by"] for la in launches)


# threads of a row's workgroup: 64 (four rows), 320 and 1024, aligned or not;
# rows that take the walking kernel
ROWS = [(1, H.HCGR_BF16), (512, H.HCGR_BF16), (2560, H.HCGR_BF16), (2559, H.HCGR_FP16), (8192, H.HCGR_BF16),
        (4096, H.HCGR_FP32), (16384, H.HCGR_BF16), (40000, H.HCGR_FP32)]


@pytest.mark.parametrize("hs,dtype", ROWS)
def test_forward_launches_of_the_longest_calls(rec, hs, dtype):
    """Below, at and above the token counts where one workgroup a row (or four
    rows) reaches 2^32 threads, and at the most tokens a call takes."""
    one_pass = hs * BYTES[dtype] <= 32 * 1024
    pieces = -(-hs * BYTES[dtype] // 16)
    edge = (1 << 32) // 64 * 4 if pieces <= 64 else (1 << 32) // min(64 * -(-pieces // 64), 1024)
    for M in (1, edge - 4, edge, edge + 4, (1 << 31) - 1, 1 << 31):
        M = min(M, 1 << 31)
        for launches in (check_sizes(norm(rec, M, hs, dtype)), check_sizes(residual(rec, M, hs, 4, dtype)),
                         check_sizes(quantize(rec, M, hs, dtype))):
            if one_pass:  # as many rows as there are tokens, whatever the launches
                assert M <= rows_of(launches) < M + 4, (M, launches)


@pytest.mark.parametrize("hs,hc,dtype", [(1, 1, H.HCGR_BF16), (2560, 4, H.HCGR_BF16), (8192, 8, H.HCGR_FP16),
                                         (16384, 2, H.HCGR_FP32)])
def test_other_launches_of_the_longest_calls(rec, hs, hc, dtype):
    for M in (1, 1 << 26, (1 << 31) - 1, 1 << 31):
        check_sizes(backward(rec, M, hs, hc, dtype))
        check_sizes(linear(rec, M, hs, 2560, dtype))
        check_sizes(linear(rec, M, hs, 16, dtype))


def combine(rec, M, hs, hc, **q):
    R, y, inj, R2 = places(M * hc * hs * 2, M * hs * 2, M * hc * 2, M * hc * hs * 2)
    return rec.ask(config="Config", values={"hc": hc, "hs": hs, "r": 32}, call="hcgr_combine",
                   args=[R, y, inj, hc, M, R2], **q)


@pytest.mark.parametrize("hs,hc", [(128, 1), (128, 4), (2560, 4), (8192, 8)])
def test_combine_launches_of_the_longest_calls(rec, hs, hc):
    edge = (1 << 32) // (256 * hc)  # a workgroup of 256 a token and stream
    for M in (1, edge - 8, edge, edge + 1, 4 * edge + 5):
        launches = check_sizes(combine(rec, M, hs, hc))
        groups = sum(la["gx"] for la in launches)
        assert M * hc <= groups < (M + 8) * hc, (M, launches)


CALLS = {"norm": lambda rec, **q: norm(rec, 100, 2560, **q), "residual": lambda rec, **q: residual(rec, 100, 512, 4, **q),
         "quantize": lambda rec, **q: quantize(rec, 100, 777, **q), "backward": lambda rec, **q: backward(rec, 100, 512, 4, **q),
         "linear": lambda rec, **q: linear(rec, 100, 2560, 512, **q)}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_handle_s_device(rec, call, current):
    """Whatever device is current: on a stream of the handle's device, or on
    that device's default stream (NULL); the caller's device stays current."""
    for device in (0, 1):
        for stream in (0, device * 16 + 3):
            a = CALLS[call](rec, device=device, current=current, stream=stream)
            assert a["status"] == H.HCGR_OK, (device, stream, a["error"])
            assert a["launches"] and a["current"] == current
            assert all(la["device"] == device and la["stream"] == stream for la in a["launches"])
        a = CALLS[call](rec, device=device, current=current, stream=(1 - device) * 16 + 3)
        assert a["status"] == H.HCGR_ERR_INVALID_ARGUMENT and "stream belongs to" in a["error"]
        assert not a["launches"] and a["current"] == current


def test_every_kernel_is_run_by_a_gpu_test(rec):
    """The shapes of the GPU tests reach every kernel of these operators that
    the library holds, so that a changed rule of choice leaves none untested."""
    import test_gpu_block as G

    def name(kernel):
        return re.sub(r"hcgr::|\(anonymous namespace\)::|^void ", "", kernel).split("(")[0]

    asked = []
    for dtype in BYTES:
        for hs, m in G.SHAPES + G.OTHER_NORM:
            asked += [norm(rec, m, hs, dtype), norm_backward(rec, m, hs, dtype)]
        for hs, m in G.OTHER_NORM:
            asked.append(quantize(rec, m, hs, dtype))
        for hc, hs, m in G.RES_SHAPES + G.OTHER_RES:
            asked += [residual(rec, m, hs, hc, dtype), backward(rec, m, hs, hc, dtype)]
        for k, m in next(p.args[1] for p in G.test_quantize.pytestmark if p.args[:1] == ("k,m",)):
            asked.append(quantize(rec, m, k, dtype))
        for n, k, m in G.LIN + G.OTHER_LIN:
            asked.append(linear(rec, m, n, k, dtype))
    run = {name(la["kernel"]) for a in asked for la in check_sizes(a)}
    held = {name(k) for k in rec.kernels()}
    held = {k for k in held if k.startswith(("norm_", "linear_"))}
    assert len(held) > 150 and not held - run, sorted(held - run)
