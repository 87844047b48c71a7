"""What making a handle of the block operators costs, and that it is enough: the
dynamic-LDS limits that it raises, recorded by a stand-in for the HIP runtime."""
import pytest

import skinny_gemm_hcgr_amd as H
import test_block_launches as T
import test_mx_launches as X
from test_block_launches import BYTES, rec  # noqa: F401

FREE = 64 * 1024  # dynamic LDS that a kernel has without asking
WIDTHS = [1, 64, 500, 512, 513, 1000, 1024, 1025, 1280, 2048, 2560, 2563, 4096, 5120, 8192, 8200, 16384, 40000, 65536]


def check(answer, most):
    """Each launch within its kernel's limit on its device, and no more limits
    raised than ``most``."""
    assert answer["status"] == H.HCGR_OK, answer["error"]
    assert len(answer["limits"]) <= most, len(answer["limits"])
    for la in answer["launches"]:
        limit = max([FREE] + [t["limit"] for t in answer["limits"] if (t["kernel"], t["device"]) == (la["kernel"], la["device"])])
        assert la["lds"] <= limit, la


@pytest.mark.parametrize("dtype", list(BYTES))
def test_block_handles(rec, dtype):  # noqa: F811
    """A handle's type and width leave two kernels of each backward pass."""
    for hs in WIDTHS:
        for m in (1, 3, 700, 100000):
            check(X.layer_norm(rec, m, hs, dtype), 4)
            check(X.layer_norm_bwd(rec, m, hs, dtype, device=1), 4)
            check(T.norm_backward(rec, m, hs, dtype), 4)
            check(T.backward(rec, m, hs, 4, dtype), 4)
            check(T.backward(rec, m, hs, 8, dtype), 4)


@pytest.mark.parametrize("dtype", list(BYTES))
def test_linear_handles(rec, dtype):  # noqa: F811
    """Of the kernels of the two products those of the handle's type."""
    for n, k in ((8, 16), (2560, 10240), (10240, 2560), (2501, 20000), (8192, 131071)):
        for m in (1, 16, 20, 32, 64, 128, 200, 512, 1024, 1400, 8192):
            check(X.linear(rec, m, n, k, dtype, device=1), 23)
            check(T.linear(rec, m, n, k, dtype), 23)
