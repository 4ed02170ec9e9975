"""Sliding windows whose passed pages have been given back: their entries of the page
table name no page any more, and attention neither follows nor reports them."""
import pytest
import torch

import test_gpu_cache as tc

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")


@pytest.fixture(scope="module")
def h():
    h = mx.mxgemm_create(0)
    yield h
    mx.mxgemm_destroy(h)


def give_back(m, news, window, sinks):
    """Entries of pages without a key that a query sees: no page, past the pages, anything."""
    given = 0
    for row, t, n in zip(m.table, m.kv_len, news):
        lo = max(0, t - n - window + 1)
        for i in range(len(row)):
            if (i + 1) * m.page <= lo and i * m.page >= sinks:
                row[i] = (-1, m.pages + 5, 2 ** 31 - 1)[given % 3]
                given += 1
    return given


@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 4), (100, 17), (130, 1), (500, 33)])
@pytest.mark.parametrize("lens,news,kv,group,d,page", [
    ([1000, 300, 41], None, 2, 4, 128, 16), ([777, 15], None, 1, 16, 64, 16), ([5000], None, 1, 8, 64, 32), ([2000, 700], None, 2, 8, 128, 128),
    ([900, 640], [3, 2], 1, 4, 64, 16), ([1100, 800], [130, 70], 4, 8, 128, 16), ([1500], [300], 8, 4, 64, 32), ([3000], [70], 1, 1, 128, 64)])
def test_passed_pages(h, lens, news, kv, group, d, page, window, sinks):
    m = tc.Made(lens, kv, d, page, seed=sum(lens))
    n = news or [1] * len(lens)
    assert give_back(m, n, window, sinks) > 0
    q = tc.queries(m, sum(n), kv * group)
    O, L = tc.attend(h, m, q, news, window=window, sinks=sinks)
    assert mx.mxgemm_get_device_status(h) == (0, 0)
    tc.check(m, q, n, O, L, window=window, sinks=sinks)


@pytest.mark.parametrize("longest", [2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1])
@pytest.mark.parametrize("lens,news", [([3, 0, 200], [7, 2, 5]), ([60, 200], [200, 130])])
def test_the_longest_windows_see_everything(h, lens, news, longest):
    """Also where a sequence has more queries than keys: the first ones stand before position 0."""
    m = tc.Made(lens, 2, 64, 16)
    q = tc.queries(m, sum(news), 4)
    want, lse = tc.attend(h, m, q, news)
    tc.check(m, q, news, want, lse)
    for window, sinks in ((longest, 0), (longest, longest), (1, longest)):
        O, L = tc.attend(h, m, q, news, window=window, sinks=sinks)
        assert torch.equal(O, want) and torch.equal(L, lse)
