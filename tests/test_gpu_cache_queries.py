"""Queries whose values differ widely within a row.

The kernels take Q in FP16 after a power of two for each row, exact down to 2^-32 of the
row's largest value and off by 2^-40 of it below; so a channel that is 2^22 times the
others, on which the keys are zero, leaves the logits as test_gpu_cache.py derives
them: values under 2^-10 of an ordinary one are off by 2^-18 of an ordinary one, which
is one value in 500."""
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


@pytest.mark.parametrize("factor", [2.0 ** 12, 2.0 ** 18, -2.0 ** 22])
@pytest.mark.parametrize("lens,news,kv,group,d,page", [
    ([300, 77], None, 2, 4, 128, 32), ([9000], None, 1, 16, 64, 64),  # single tokens, 8 and 16 rows an item
    ([300, 250], [200, 100], 8, 4, 128, 64), ([700], [300], 2, 2, 64, 16)])  # prompts
def test_one_large_channel(h, lens, news, kv, group, d, page, factor):
    m = tc.Made(lens, kv, d, page, seed=sum(lens))
    used = m.K != 0x7F
    m.K[..., 5] = torch.where(used[..., 5], 0, m.K[..., 5])  # (NaN codes stay where no key is)
    n = news or [1] * len(lens)
    q = tc.queries(m, sum(n), kv * group)
    q[..., 5] = (q[..., 6].float().abs().clamp(min=0.25) * factor).bfloat16()
    O, L = tc.attend(h, m, q, news)
    tc.check(m, q, n, O, L)


@pytest.mark.parametrize("news", [None, [70, 100]])
def test_queries_at_the_ends_of_their_type(h, news):
    """Rows whose largest value is BF16's largest or among its smallest, and rows of zeros."""
    m = tc.Made([180, 250], 2, 128, 16)
    n = news or [1, 1]
    top = 3.3895313892515355e38
    for f, scale in ((top, 0.05 / top), (2.0 ** -110, 0.05 * 2.0 ** 110), (2.0 ** -126, 0.05 * 2.0 ** 126)):
        q = (tc.queries(m, sum(n), 8).float().clamp(-1, 1) * f).bfloat16()
        q[0, 0, 3] = f
        q[0, 1] = 0
        O, L = tc.attend(h, m, q, news, scale=scale)
        tc.check(m, q, n, O, L, scale=scale)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,news,kv,group,d,page", [
    ([300, 77], None, 2, 4, 128, 32), ([9000, 64], None, 1, 16, 64, 64), ([20011], None, 1, 8, 128, 64),  # whole, split
    ([300, 250], [200, 100], 8, 4, 128, 64), ([5000], [70], 1, 1, 128, 64)])  # prompts, the second with its keys cut
def test_nan_stays_in_its_row(h, lens, news, kv, group, d, page, value):
    """A query that is not finite gives a NaN output and log-sum-exp, and no other row one."""
    m = tc.Made(lens, kv, d, page, seed=sum(lens))
    n = news or [1] * len(lens)
    q = tc.queries(m, sum(n), kv * group)
    want, lse = tc.attend(h, m, q, news)
    bad = torch.zeros(sum(n), kv * group, dtype=torch.bool)
    bad[0, 0] = bad[-1, -1] = True
    q[0, 0] = value if value != value else q[0, 0]
    q[0, 0, 1] = q[-1, -1, 1] = value
    O, L = tc.attend(h, m, q, news)
    assert torch.isnan(O[bad]).all() and torch.isnan(L[bad]).all()
    assert torch.equal(O[~bad], want[~bad]) and torch.equal(L[~bad], lse[~bad])
