"""Attention of sequences that share their first tokens, on the GPU: against the plain
64-bit implementation, with the tolerances of tests/test_gpu_cache.py (the shared part
and the own part are joined in FP32, which adds 2^-22 of the sums), whatever part of the
tokens the call is told to be shared."""
import math

import pytest
import torch

import plain64
from test_gpu_cache import DEV, Made, check, mx, queries, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    """A handle that reads the shared keys apart whatever their number."""
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_SHARED_KEYS, 1)
    yield h
    mx.mxgemm_destroy(h)


def made(lens, kv, d, page, common, seed=0, **kw):
    """Sequences whose tables agree on the pages of the first `common` tokens, as far as
    they reach; what no sequence holds is NaN codes."""
    m = Made(lens, kv, d, page, seed=seed, **kw)
    longest = max(range(len(lens)), key=lambda i: lens[i])
    for row in m.table:
        n = min(len(row), common // page)
        row[:n] = m.table[longest][:n]
    return m


def attend(h, m, q, news, shared, scale=None, stream=None, causal=True, lse=True):
    tokens, heads, _ = q.shape
    cache, table = m.cache(), m.table_tensor()
    lens = torch.tensor(m.kv_len, dtype=torch.int32, device=DEV)
    starts = None if news is None else torch.tensor(starts_of(news), dtype=torch.int32, device=DEV)
    O = torch.full((tokens, heads, m.d), math.nan, dtype=torch.bfloat16, device=DEV)
    L = torch.full((tokens, heads), math.nan, device=DEV) if lse else None
    mx.mxgemm_cache_attention_shared(h, cache, table, lens, shared, q if q.is_cuda else q.to(DEV), O, q_start=starts, scale=scale, causal=causal,
                                     lse=L, stream=stream)
    torch.cuda.synchronize()
    return O.cpu(), None if L is None else L.cpu()


TOKENS = [  # lengths, shared tokens, kv heads, heads of a group, d, page
    ([65, 70, 90], 64, 1, 1, 128, 16), ([200, 129, 300, 129], 128, 2, 4, 64, 32), ([1000] * 5, 512, 1, 8, 128, 64),
    ([600, 0, 513, 40], 512, 2, 7, 128, 64), ([2049, 2500], 2048, 2, 16, 128, 128), ([700] * 40, 640, 2, 4, 64, 128),
    ([5000, 4097, 4100], 4096, 1, 40, 128, 16), ([300, 300], 288, 3, 2, 128, 16), ([3, 1, 2], 0, 1, 4, 128, 16), ([900] * 70, 800, 1, 1, 128, 32),
]


@pytest.mark.parametrize("lens,common,kv,group,d,page", TOKENS)
def test_single_tokens(h, lens, common, kv, group, d, page):
    m = made(lens, kv, d, page, common, seed=sum(lens))
    q = queries(m, len(lens), kv * group)
    # all of the common tokens, a part of a page less, one page, more than there is, none
    for shared in {common, max(0, common - 5), page, common + page - 1, 0}:
        O, L = attend(h, m, q, None, shared)
        check(m, q, [1] * len(lens), O, L)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


SEVERAL = [  # lengths, new tokens, shared tokens, kv heads, group, d, page
    ([70, 90, 65], [4, 4, 1], 64, 2, 4, 128, 16), ([300, 200, 260], [40, 3, 0], 160, 1, 8, 64, 32), ([700, 600, 520], [180, 80, 5], 512, 4, 2, 128, 64),
    ([1500, 1300], [400, 257], 1024, 2, 4, 128, 128), ([400, 64, 130], [300, 64, 2], 128, 2, 7, 128, 64), ([0, 500, 100], [2, 130, 100], 96, 1, 3, 64, 16),
    ([2000] * 6, [16] * 6, 1900 // 16 * 16, 8, 4, 128, 16),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,news,common,kv,group,d,page", SEVERAL)
def test_several_tokens(h, lens, news, common, kv, group, d, page, causal):
    """Drafts and prompts; tokens whose own positions lie within the shared ones too."""
    m = made(lens, kv, d, page, common, seed=sum(lens))
    q = queries(m, sum(news), kv * group)
    for shared in {common, page}:
        O, L = attend(h, m, q, news, shared, causal=causal)
        check(m, q, news, O, L, causal=causal)
        again, L2 = attend(h, m, q, news, shared, causal=causal)
        assert torch.equal(O, again) and torch.equal(L, L2)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


def test_as_without_sharing(h):
    """The call without sharing, on the same tables: within both tolerances."""
    lens = [1200, 1025, 1100]
    m = made(lens, 2, 128, 64, 1024)
    q = queries(m, 3, 16)
    O, L = attend(h, m, q, None, 1024)
    O0 = torch.empty(3, 16, 128, dtype=torch.bfloat16, device=DEV)
    L0 = torch.empty(3, 16, device=DEV)
    mx.mxgemm_cache_attention(h, m.cache(), m.table_tensor(), torch.tensor(lens, dtype=torch.int32, device=DEV), q.to(DEV), O0, lse=L0)
    torch.cuda.synchronize()
    _, _, mag, size = plain64.attention(plain64.value(m.K), m.sK, plain64.value(m.V), m.sV, m.table, lens, [0, 1, 2, 3], q, 128 ** -0.5)
    assert ((O.double() - O0.cpu().double()).abs() <= 2.0 ** -7 * O.double().abs() + 2.0 ** -9 * mag).all()
    assert ((L.double() - L0.cpu().double()).abs() <= 2.0 ** -18 * (1 + size)).all()


def test_chosen_by_the_library():
    """Few shared keys are read with each sequence's own, as the call without sharing
    does it (equal bits, one launch); many apart (three launches)."""
    h = mx.mxgemm_create(0)
    with pytest.raises(mx.MxgemmError):
        mx.mxgemm_set_option(h, mx.OPT_SHARED_KEYS, 2)
    m = made([200, 190], 2, 128, 16, 128)
    q = queries(m, 2, 8)
    n = mx.mxgemm_get_launch_count(h)
    O, L = attend(h, m, q, None, 128)
    assert mx.mxgemm_get_launch_count(h) == n + 1
    O0, L0 = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(2, 8, device=DEV)
    mx.mxgemm_cache_attention(h, m.cache(), m.table_tensor(), torch.tensor(m.kv_len, dtype=torch.int32, device=DEV), q.to(DEV), O0, lse=L0)
    torch.cuda.synchronize()
    assert torch.equal(O, O0.cpu()) and torch.equal(L, L0.cpu())
    m = made([4100 + i for i in range(96)], 2, 128, 64, 4096)
    q = queries(m, 96, 4)
    n = mx.mxgemm_get_launch_count(h)
    O, L = attend(h, m, q, None, 4096)
    assert mx.mxgemm_get_launch_count(h) == n + 3
    check(m, q, [1] * 96, O, L)
    assert mx.mxgemm_get_device_status(h) == (0, 0)
    mx.mxgemm_destroy(h)


@pytest.mark.parametrize("f,scale", [(2.0 ** 20, 0.08), (2.0 ** -40, 0.08), (1.0, -0.1)])
def test_wide_scales(h, f, scale):
    """Page scales over 2^30, queries past FP16's range, a negative scale."""
    m = made([300, 290, 270], 2, 128, 16, 256, scales=(-30, 0))
    m.sK.fill_(2.0 ** -8)
    q = (queries(m, 3, 8).float() * f).bfloat16()
    O, L = attend(h, m, q, None, 256, scale=scale / f)
    check(m, q, [1] * 3, O, L, scale=scale / f)


def test_one_part_outweighs_the_other(h):
    """Keys of one part thousands of times the other's weight, either way round: logits 40 apart."""
    for own in (False, True):
        m = made([192, 180, 150], 1, 64, 16, 128)
        at = torch.tensor(sorted({p for row in m.table for i, p in enumerate(row) if (i >= 8) == own}))
        m.sK[at] *= 8
        q = queries(m, 3, 4)
        O, L = attend(h, m, q, None, 128)
        check(m, q, [1] * 3, O, L)


def test_bad_pages_and_lengths(h):
    """Page numbers that name no page and lengths that do not fit are recorded and not followed."""
    m = made([200, 180, 190], 1, 128, 16, 128)
    m.table[0][2] = m.table[1][2] = m.table[2][2] = m.pages + 5
    q = queries(m, 3, 8)
    O, L = attend(h, m, q, None, 128)
    check(m, q, [1] * 3, O, L)
    assert mx.mxgemm_get_device_status(h) == (mx.ERR_INVALID_VALUE, 0x23)
    m = made([200, 180, 190], 1, 128, 16, 128)
    cache, table = m.cache(), m.table_tensor()
    O = torch.full((3, 8, 128), math.nan, dtype=torch.bfloat16, device=DEV)
    mx.mxgemm_cache_attention_shared(h, cache, table, torch.tensor([200, 10 ** 6, 190], dtype=torch.int32, device=DEV), 128, q.to(DEV), O)
    torch.cuda.synchronize()
    assert mx.mxgemm_get_device_status(h) == (mx.ERR_INVALID_VALUE, 0x21)
    want, _ = attend(h, m, q, None, 128)
    O = O.cpu()
    assert (O[1] == 0).all() and torch.equal(O[0], want[0]) and torch.equal(O[2], want[2])


def test_rows_of_padding(h):
    """Sequences without tokens in a padded batch: zeros, whatever their row of the table says, the first among them."""
    lens = [0, 300, 0, 260]
    m = made(lens, 2, 128, 64, 256)
    q = queries(m, 4, 8)
    O, L = attend(h, m, q, None, 256)
    check(m, q, [1] * 4, O, L)
    m2 = made([0, 0], 2, 128, 64, 0)
    O, L = attend(h, m2, queries(m2, 2, 8), None, 128)
    assert (O == 0).all() and (L == -math.inf).all()
    assert mx.mxgemm_get_device_status(h) == (0, 0)


@pytest.mark.parametrize("new", [1, 3])
def test_more_shared_tokens_than_any_sequence_has(h, new):
    """All sequences within the shared tokens: nothing of their own is left, and a
    length past all of them is no longer than the table."""
    m = made([200, 130, 64], 2, 128, 16, 10 ** 6)
    q = queries(m, 3 * new, 8)
    for shared in (208, 10 ** 6, 2 ** 40):
        O, L = attend(h, m, q, [new] * 3, shared)
        check(m, q, [new] * 3, O, L)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


def test_refusals(h):
    m = made([64, 64], 1, 64, 16, 32)
    cache, table, lens = m.cache(), m.table_tensor(), torch.tensor([64, 64], dtype=torch.int32, device=DEV)
    q = queries(m, 2, 3).to(DEV)
    O = torch.empty_like(q)
    call = lambda shared, **kw: mx.mxgemm_cache_attention_shared(h, cache, table, lens, shared, q, O, check=False, **kw)  # noqa: E731
    assert call(-1) == mx.ERR_INVALID_VALUE
    assert call(32, scale=math.nan) == mx.ERR_INVALID_VALUE
    assert call(32) == mx.OK
    torch.cuda.synchronize()


def test_rows_behind_the_last_sequence_stay(h):
    m = made([200, 190], 1, 128, 16, 128)
    q = queries(m, 6, 4)
    cache, table = m.cache(), m.table_tensor()
    O = torch.full((6, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    starts = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    mx.mxgemm_cache_attention_shared(h, cache, table, torch.tensor([200, 190], dtype=torch.int32, device=DEV), 128, q.to(DEV), O, q_start=starts)
    torch.cuda.synchronize()
    assert (O[4:] == 7).all()
    check(m, q[:4], [2, 2], O[:4].cpu(), None)


def test_graph_with_growing_sequences(h):
    """A captured step replayed with other lengths, queries and table."""
    m = made([256, 250, 240], 2, 128, 16, 128)
    cache, table, every = m.cache(), m.table_tensor(), m.table
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    q, O = torch.zeros(3, 16, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 16, 128, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mxgemm_cache_attention_shared(h, cache, table, lens, 128, q, O, stream=torch.cuda.current_stream())
    for n in ([200, 180, 190], [201, 181, 130], [129, 250, 131], [0, 256, 100], [100, 90, 7]):
        n = [min(x, y) for x, y in zip(n, (256, 250, 240))]
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        q.copy_(queries(m, 3, 16, seed=n[0]))
        graph.replay()
        torch.cuda.synchronize()
        m.kv_len, m.table = n, [row[:-(-t // 16)] for row, t in zip(every, n)]
        check(m, q.cpu(), [1] * 3, O.cpu(), None)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


@pytest.mark.parametrize("new", [1, 16])
@pytest.mark.parametrize("copies", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_reads_what_was_appended_just_before(h, new, graph, copies):
    """The launch over the own keys does not wait for the one before it: steps in a row,
    in which the pages' codes and scales, the lengths and the queries change, give what
    they give with the device idle between any two calls, to the bit.  With the steps'
    inputs in buffers of their own, or copied into the same ones."""
    batch, steps, kv, group, d, page, common = 24, 8, 2, 4, 128, 16, 512
    m = made([common + 20 + steps * new + i for i in range(batch)], kv, d, page, common, seed=3)
    table = m.table_tensor()
    g = torch.Generator().manual_seed(4)
    K, V = ((torch.randn(steps, batch * new, kv, d, generator=g) * 1.5 ** torch.arange(steps).view(-1, 1, 1, 1)).bfloat16().to(DEV) for _ in range(2))
    Q = torch.randn(steps, batch * new, kv * group, d, generator=g).bfloat16().to(DEV)
    lens = torch.tensor([[n - (steps - 1 - i) * new for n in m.kv_len] for i in range(steps)], dtype=torch.int32, device=DEV)
    starts = torch.arange(batch + 1, dtype=torch.int32, device=DEV) * new if new > 1 else None

    def run(cache, q, k, v, n, O, wait):
        for i in range(steps):
            if copies:
                for to, what in ((q, Q), (k, K), (v, V), (n, lens)):
                    to.copy_(what[i])
            else:
                q, k, v, n = Q[i], K[i], V[i], lens[i]
            wait()
            mx.mxgemm_cache_append(h, cache, table, n, k, v, q_start=starts, stream=torch.cuda.current_stream())
            wait()
            mx.mxgemm_cache_attention_shared(h, cache, table, n, common, q, O[i], q_start=starts, stream=torch.cuda.current_stream())
            wait()

    def buffers():
        return (m.cache(), *(torch.empty_like(x[0]) for x in (Q, K, V, lens)), torch.full_like(Q, math.nan))

    want = buffers()
    run(*want, torch.cuda.synchronize)
    got = buffers()
    if graph:
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            run(*got, lambda: None)
        cg.replay()
    else:
        run(*got, lambda: None)
    torch.cuda.synchronize()
    assert torch.isfinite(want[5].float()).all() and torch.equal(got[5], want[5])
    assert mx.mxgemm_get_device_status(h) == (0, 0)


@pytest.mark.parametrize("new", [1, 40])
def test_a_call_that_gives_up_leaves_nothing(new):
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_SHARED_KEYS, 1)
    lens, news = [700, 650, 600], [new] * 3
    m = made(lens, 2, 128, 16, 512)
    q = queries(m, 3 * new, 16)
    want, _ = attend(h, m, q, news, 512)
    mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000)
    mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, 1)
    attend(h, m, q, news, 512)
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_TIMEOUT
    mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, 0)
    mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
    again, _ = attend(h, m, q, news, 512)
    assert torch.equal(want, again) and mx.mxgemm_get_device_status(h) == (0, 0)
    mx.mxgemm_destroy(h)


def test_two_handles_on_two_streams(h):
    """The same batch on two streams at once, each with its handle: equal bits."""
    other = mx.mxgemm_create(0)
    mx.mxgemm_set_option(other, mx.OPT_SHARED_KEYS, 1)
    m = made([3000] * 8, 2, 128, 64, 2560)
    q = queries(m, 8, 16).to(DEV)
    want, _ = attend(h, m, q, None, 2560)
    cache, table, lens = m.cache(), m.table_tensor(), torch.tensor(m.kv_len, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros(8, 16, 128, dtype=torch.bfloat16, device=DEV) for _ in range(6)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(6):
        for handle, side, out in zip((h, other), sides, outs):
            mx.mxgemm_cache_attention_shared(handle, cache, table, lens, 2560, q, out[i], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for out in outs for o in out)
    mx.mxgemm_destroy(other)
