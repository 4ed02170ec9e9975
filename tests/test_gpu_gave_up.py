"""Calls whose waits give up: they end with a status, and the handle works as
before afterwards.  The test hook keeps loads from being issued; where one CTA of a
pair stops alone, what the other has loaded lands long before the waits run out."""
import pytest
import torch

import plain64
import test_gpu_block128 as tb
import test_gpu_cache as tc

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")


@pytest.fixture
def h():
    h = mx.mxgemm_create(0)
    yield h
    mx.mxgemm_destroy(h)


class Stalled:
    """Short waits, and loads held back as `how` says."""

    def __init__(self, h, how=1):
        self.h, self.how = h, how

    def __enter__(self):
        mx.mxgemm_set_option(self.h, mx.OPT_WAIT_TIMEOUT_NS, 20_000_000)
        mx.mxgemm_set_option(self.h, mx.OPT_TEST_STALL_PRODUCER, self.how)

    def __exit__(self, *_):
        mx.mxgemm_set_option(self.h, mx.OPT_TEST_STALL_PRODUCER, 0)
        mx.mxgemm_set_option(self.h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000_000)


# whole items, items of several CTAs, both counts of rows an item
@pytest.mark.parametrize("lens,kv,group,d,page", [([100, 40], 1, 4, 128, 16), ([20011, 64], 1, 8, 128, 64), ([3000, 700], 2, 16, 64, 32)])
def test_single_tokens(h, lens, kv, group, d, page):
    m = tc.Made(lens, kv, d, page)
    q = tc.queries(m, len(lens), kv * group)
    want, lse = tc.attend(h, m, q, None)
    tc.check(m, q, [1] * len(lens), want, lse)
    with Stalled(h):
        tc.attend(h, m, q, None)
    for _ in range(2):  # before and after the status is read
        O, L = tc.attend(h, m, q, None)
        assert torch.equal(O, want) and torch.equal(L, lse)
        status, detail = mx.mxgemm_get_device_status(h)
        assert (status, detail) == ((mx.ERR_TIMEOUT, 0x31) if _ == 0 else (0, 0))


# row tiles with a CTA each, and row tiles whose keys are cut into parts
@pytest.mark.parametrize("lens,news,kv,group,d,page", [([1100], [1100], 4, 4, 128, 64), ([400], [257], 160, 3, 64, 128),
                                                       ([5000], [70], 1, 1, 128, 64), ([3001, 0, 129], [40, 2, 100], 1, 8, 64, 32)])
def test_prompts(h, lens, news, kv, group, d, page):
    m = tc.Made(lens, kv, d, page)
    q = tc.queries(m, sum(news), kv * group)
    want, lse = tc.attend(h, m, q, news)
    tc.check(m, q, news, want, lse)
    with Stalled(h):
        tc.attend(h, m, q, news)
    for read in (0, 1):
        O, L = tc.attend(h, m, q, news)
        assert torch.equal(O, want) and torch.equal(L, lse)
        status, detail = mx.mxgemm_get_device_status(h)
        assert (status == mx.ERR_TIMEOUT and 0x41 <= detail <= 0x4F) if read == 0 else (status, detail) == (0, 0)


# the CTAs of a pair stop at different loads: what one of them has issued alone lands before the pair ends
@pytest.mark.parametrize("how", [1, 2, 3])
@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("m,n,k,b_block", [(300, 304, 400, 128), (300, 304, 1200, 1), (2100, 2304, 1680, 128)])
def test_products(h, m, n, k, b_block, nk, how):
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K if nk else mx.B_K_BY_N)
    a, sa, b, sb = tb.operands(m, n, k, b_block, 1)
    ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, b_block)
    if not nk:
        b, sb = b.t().contiguous(), sb.t().contiguous()
    dev = [t.to(tb.DEV) for t in (a, sa, b, sb)]
    C = torch.zeros(m, n, device=tb.DEV)
    with Stalled(h, how):
        mx.mxgemm_run_block128(h, m, n, k, *dev, C, b_block=b_block)
        assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_TIMEOUT
    mx.mxgemm_run_block128(h, m, n, k, *dev, C, b_block=b_block)
    assert mx.mxgemm_get_device_status(h) == (0, 0)
    tb.check(C.cpu(), ref, mag, "f32")


@pytest.mark.parametrize("m,n,k", [(300, 300, 4096), (300, 304, 6416), (2600, 2304, 4096)])
@pytest.mark.parametrize("hidden", [False, True])
def test_tiles_cut_along_k(h, m, n, k, hidden):
    """One part of a tile whose K is cut gives up, the others are done: later calls
    do not take what is left of it for theirs, be its status read, hidden behind an
    earlier one, or not read yet."""
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
    a, sa, b, sb = tb.operands(m, n, k, 128, 1)
    ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, 128)
    dev = [t.to(tb.DEV) for t in (a, sa, b, sb)]
    C = torch.zeros(m, n, device=tb.DEV)
    call = lambda: mx.mxgemm_run_block128(h, m, n, k, *dev, C)
    call()
    want = C.cpu()
    tb.check(want, ref, mag, "f32")
    for read in (True, False):
        if hidden:  # a page number that names no page
            pages = tc.Made([40], 1, 64, 16)
            pages.table[0][1] = -1
            tc.attend(h, pages, tc.queries(pages, 1, 1), None)
        with Stalled(h, 4):
            call()
        if read:
            assert mx.mxgemm_get_device_status(h)[0] == (mx.ERR_INVALID_VALUE if hidden else mx.ERR_TIMEOUT)
        other = [t.flip(0).contiguous() for t in dev]  # other sums than the ones that were left
        mx.mxgemm_run_block128(h, m, n, k, *other, C)
        for _ in range(2):
            C.zero_()
            call()
            assert torch.equal(C.cpu(), want)
        if not read:
            mx.mxgemm_get_device_status(h)
    assert mx.mxgemm_get_device_status(h) == (0, 0)
