"""Attention behind shared tokens with page tables far wider than the sequences, as a
captured step has them: what is shared is read apart all the same, and the results are
right whether the sequences' own keys are few or many (tolerances of
tests/test_gpu_cache.py)."""
import pytest
import torch

from test_gpu_cache import DEV, check, mx, queries
from test_gpu_shared import attend, made

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    h = mx.mxgemm_create(0)
    yield h
    mx.mxgemm_destroy(h)


@pytest.mark.parametrize("room", [0, 16384, 65536, 2 ** 20])
@pytest.mark.parametrize("batch,kv,group,page,new", [(96, 2, 2, 64, 1), (64, 4, 8, 128, 1), (24, 2, 4, 16, 4)])
def test_the_tables_width_does_not_decide(h, batch, kv, group, page, new, room):
    m = made([4100 + 3 * i for i in range(batch)], kv, 128, page, 4096)
    m.width = max(m.width, room // page)
    q = queries(m, batch * new, kv * group)
    news = None if new == 1 else [new] * batch
    n = mx.mxgemm_get_launch_count(h)
    O, L = attend(h, m, q, news, 4096)
    assert mx.mxgemm_get_launch_count(h) == n + 3
    check(m, q, [new] * batch, O, L)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


@pytest.mark.parametrize("d,group,new", [(128, 4, 1), (128, 16, 1), (64, 4, 2)])
def test_replayed_with_few_and_with_many_own_keys(d, group, new):
    """One captured step whose sequences have one own key, some, and thousands: on the SMs
    beside the shared keys' launch, and on all.  (Apart whatever the estimates say.)"""
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_SHARED_KEYS, 1)
    batch, common, page, longest = 12, 1024, 64, 9000
    m = made([longest - 50 * i for i in range(batch)], 2, d, page, common)
    m.width = 32768 // page
    cache, table, every = m.cache(), m.table_tensor(), m.table
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    starts = torch.arange(batch + 1, dtype=torch.int32, device=DEV) * new
    q = torch.zeros(batch * new, 2 * group, d, dtype=torch.bfloat16, device=DEV)
    O = torch.zeros_like(q)
    n = mx.mxgemm_get_launch_count(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mxgemm_cache_attention_shared(h, cache, table, lens, common, q, O, q_start=starts, stream=torch.cuda.current_stream())
    assert mx.mxgemm_get_launch_count(h) == n + 3
    for own in (1, 40, 700, longest - common, 5):
        now = [max(new, min(common + own - i, longest - 50 * i)) for i in range(batch)]
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(queries(m, batch * new, 2 * group, seed=own))
        graph.replay()
        torch.cuda.synchronize()
        m.kv_len, m.table = now, [row[:-(-t // page)] for row, t in zip(every, now)]
        check(m, q.cpu(), [new] * batch, O.cpu(), None)
    assert mx.mxgemm_get_device_status(h) == (0, 0)
    mx.mxgemm_destroy(h)
