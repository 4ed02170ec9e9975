"""Scales of the block-128 product near the ends of the range that mxgemm.h states for
them.  Tolerance as in test_gpu_block128.py: 1e-5 of the sum of the terms'
magnitudes."""
import pytest
import torch

import plain64
import test_gpu_block128 as tb

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")


@pytest.fixture(scope="module")
def handles():
    hs = {}
    for nk in (True, False):
        hs[nk] = mx.mxgemm_create(0)
        mx.mxgemm_set_option(hs[nk], mx.OPT_B_MAJOR, mx.B_N_BY_K if nk else mx.B_K_BY_N)
    yield hs
    for h in hs.values():
        mx.mxgemm_destroy(h)


def smallest(shape, g):
    """Codes 0 to 3 times 2^-9."""
    return torch.randint(0, 4, shape, generator=g).to(torch.uint8)


# exponents of the scales of A and of B, and codes: scale products just in FP32's
# normal range (a factor of 2 for each scale's own spread is left), and scales that
# are far out while their product is not
CASES = {"small": (-84, -40, tb.random_codes), "large": (88, 38, smallest), "opposite": (-80, 80, tb.random_codes),
         "other way": (80, -80, tb.random_codes)}


@pytest.mark.parametrize("b_block", [128, 1])
@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("m", [5, 30, 64, 300])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("mixed", [False, True])
def test_scales_at_the_ends_of_their_range(handles, case, m, nk, b_block, mixed):
    ea, eb, codes = CASES[case]
    n, k = 304, 1168
    a, sa, b, sb = tb.operands(m, n, k, b_block, m, codes)
    sa, sb = sa.clamp(0.5, 1.9) * 2.0 ** ea, sb.clamp(0.5, 1.9) * 2.0 ** eb
    if mixed:  # every other row, and every third K block of B, are ordinary or meet in the middle
        sa[::2] *= 2.0 ** (-ea // 2)
        sb[:, ::3] *= 2.0 ** (-eb // 2)
    ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, b_block)
    assert float(mag.min()) > 2.0 ** -126 and float(mag.max()) < 2.0 ** 127
    tb.check(tb.run(handles[nk], nk, a, sa, b, sb, b_block), ref, mag, "f32")
