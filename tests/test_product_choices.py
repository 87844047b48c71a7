"""Which kernel of the microscaled product the GPU tests' shapes take, recorded by
a stand-in for the HIP runtime: short and deep rows on each kernel, and parts of
a batch on the kernel of the whole."""
import re

import pytest

from test_block_launches import BYTES, check_sizes, rec  # noqa: F401
from test_mx_launches import linear


def kernel(rec, n, k, m, dtype):  # noqa: F811
    la, = check_sizes(linear(rec, m, n, k, dtype))
    return re.sub(r"hcgr::|\(anonymous namespace\)::|^void ", "", la["kernel"]).split("(")[0], la["bx"]


@pytest.mark.parametrize("dtype", list(BYTES))
def test_each_kernel_runs_with_short_and_with_deep_rows(rec, dtype):  # noqa: F811
    import test_gpu_mx as G
    import test_gpu_mx_invariants as I
    kinds = {kernel(rec, *s, dtype)[0] for s in G.LIN}
    short = {kernel(rec, *s, dtype)[0] for s in G.LIN if s[1] <= 16384}
    deep = {kernel(rec, *s, dtype)[0] for s in I.DEEP}
    assert all(k > 16384 for _, k, _ in I.DEEP)
    assert len(kinds) == 11 and short == kinds and deep == kinds, (kinds - short, kinds - deep)


def test_a_large_bias_meets_each_kernel(rec):  # noqa: F811
    import test_gpu_mx_invariants as I
    from skinny_gemm_hcgr_amd import HCGR_FP32
    assert len({kernel(rec, *s, HCGR_FP32)[0] for s in I.BIAS}) == 11


@pytest.mark.parametrize("dtype", list(BYTES))
def test_parts_of_a_batch_take_its_kernel(rec, dtype):  # noqa: F811
    import test_gpu_mx_invariants as I
    for n, k, m, (a, z) in I.PARTS:
        assert kernel(rec, n, k, m, dtype) == kernel(rec, n, k, z - a, dtype), (n, k, m)
