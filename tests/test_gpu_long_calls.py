"""Calls that take longer than the limit of their waits: no role may count the time in
which another is at work as a wait that ran out."""
import pytest
import torch

import plain64
import test_gpu_block128 as tb

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"


def test_product_of_more_than_two_seconds():
    """147456 cubed: 6.4e15 operations, more than the two seconds that the waits at a
    kernel's end have, with a limit of 20 ms for the others."""
    if torch.cuda.mem_get_info()[0] < 120 * 2 ** 30:
        pytest.skip("needs 100 GB")
    n = 147456
    g = torch.Generator(device=DEV).manual_seed(1)
    a, b = (torch.randint(0, 0x7F, (n, n), generator=g, dtype=torch.uint8, device=DEV) for _ in range(2))
    sa, sb = torch.rand(n, n // 128, generator=g, device=DEV) + 0.5, torch.rand(n // 128, n // 128, generator=g, device=DEV) + 0.5
    C = torch.empty(n, n, dtype=torch.bfloat16, device=DEV)
    h = mx.mxgemm_create(0)
    try:
        mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
        mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 20_000_000)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        mx.mxgemm_run_block128(h, n, n, n, a, sa, b, sb, C, out_dtype=mx.OUT_BF16)
        end.record()
        assert mx.mxgemm_get_device_status(h) == (0, 0)
        assert begin.elapsed_time(end) > 2000
        rows, cols = torch.tensor([0, 70001, n - 1], device=DEV), torch.tensor([0, 255, 256, 100003, n - 1], device=DEV)
        A, B = a[rows].cpu(), b[cols].cpu()
        ref, mag = plain64.product(plain64.value(A), sa[rows].cpu(), plain64.value(B), sb[cols // 128].cpu(), 1)
        tb.check(C[rows][:, cols].cpu(), ref, mag, "bf16")
    finally:
        mx.mxgemm_destroy(h)
