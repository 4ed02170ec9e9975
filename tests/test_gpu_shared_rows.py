"""Attention behind shared tokens where some rows of the queries are no sequence's: a batch
that is padded in tokens, before its first sequence or behind its last, or with starts
that are refused.  Such rows stay as they were, whatever earlier calls left in the
handle's workspace; the others are right (tolerances of tests/test_gpu_cache.py)."""
import pytest
import torch

import plain64
from test_gpu_cache import DEV, Made, mx, queries
from test_gpu_shared import made

pytestmark = pytest.mark.gpu


@pytest.fixture
def h():
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_SHARED_KEYS, 1)
    yield h
    mx.mxgemm_destroy(h)


def fill_workspace(h):
    """A larger call, all of whose sums are positive: read as whole numbers they are some 10^9."""
    m = made([4200] * 48, 2, 128, 64, 4096, seed=9)
    m.V = torch.where(m.V == 0x7F, m.V, m.V & 0x7F)
    q = queries(m, 48, 32).to(DEV)
    mx.mxgemm_cache_attention_shared(h, m.cache(), m.table_tensor(), torch.tensor(m.kv_len, dtype=torch.int32, device=DEV), 4096, q, torch.empty_like(q))


def attend(h, m, q, starts, shared):
    O = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    L = torch.full(q.shape[:2], 7.0, device=DEV)
    mx.mxgemm_cache_attention_shared(h, m.cache(), m.table_tensor(), torch.tensor(m.kv_len, dtype=torch.int32, device=DEV), shared, q.to(DEV), O,
                                     q_start=torch.tensor(starts, dtype=torch.int32, device=DEV), lse=L)
    torch.cuda.synchronize()
    return O.cpu(), L.cpu()


def check(m, q, starts, O, L, whose, maybe=False):
    """whose: the sequence of each row, -1 for none.  Sequences without a row are left
    out, and, with `maybe`, rows that were."""
    for b in range(len(m.kv_len)):
        rows = [t for t, s in enumerate(whose) if s == b]
        if not rows or maybe and (O[rows] == 7).all() and (L[rows] == 7).all():
            continue
        o, lse, mag, size = plain64.attention(plain64.value(m.K), m.sK, plain64.value(m.V), m.sV, m.table[b:b + 1], m.kv_len[b:b + 1], [0, len(rows)],
                                              q[rows], m.d ** -0.5)
        assert float(size.max()) < 64
        assert ((O[rows].double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -10 * mag).all()
        assert ((L[rows].double() - lse).abs() <= 2.0 ** -19 * (1 + size)).all()
    none = torch.tensor([s < 0 for s in whose])
    assert (O[none] == 7).all() and (L[none] == 7).all()


GAPS = [  # starts, tokens, refused sequences
    ([3, 4, 6, 9], 9, ()),  # before the first
    ([0, 2, 3, 6], 11, ()),  # behind the last
    ([5, 6, 6, 8], 20, ()),  # both, and a sequence without rows
    ([0, 3, -1, 8], 9, (1, 2)), ([0, 2, 30, 9], 9, (1, 2)), ([40, 41, 4, 6], 9, (0, 1)),  # refused
]


@pytest.mark.parametrize("shared", [96, 512])
@pytest.mark.parametrize("group", [4, 16, 40])
@pytest.mark.parametrize("starts,tokens,refused", GAPS)
def test_rows_of_no_sequence_stay(h, starts, tokens, refused, group, shared):
    m = made([shared + 60, shared + 9, shared + 200], 2, 128, 32, shared, seed=group)
    q = queries(m, tokens, 2 * group)
    whose = [-1] * tokens
    for b in range(3):
        if b not in refused:
            whose[starts[b]:starts[b + 1]] = [b] * (starts[b + 1] - starts[b])
    fill_workspace(h)
    O, L = attend(h, m, q, starts, shared)
    check(m, q, starts, O, L, whose, bool(refused))
    assert mx.mxgemm_get_device_status(h) == ((mx.ERR_INVALID_VALUE, 0x22) if refused else (0, 0))


def test_padded_prompts(h):
    """Many rows of a sequence (the other kernel), with rows before, behind and more row tiles of padding alone."""
    starts, tokens = [70, 170, 270], 900
    m = made([300, 240], 2, 64, 16, 128)
    q = queries(m, tokens, 8)
    fill_workspace(h)
    O, L = attend(h, m, q, starts, 128)
    check(m, q, starts, O, L, [-1] * 70 + [0] * 100 + [1] * 100 + [-1] * 630)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


def test_no_row_is_a_sequences(h):
    m = made([200, 190], 1, 128, 16, 128)
    q = queries(m, 6, 4)
    fill_workspace(h)
    O, L = attend(h, m, q, [4, 4, 4], 128)
    assert (O == 7).all() and (L == 7).all()


@pytest.mark.parametrize("starts,tokens", [([3, 4, 6], 9), ([100, 200, 300], 400)])
def test_rows_stay_when_a_call_gives_up(h, starts, tokens):
    m = made([700, 650], 2, 128, 16, 512)
    q = queries(m, tokens, 8)
    fill_workspace(h)
    torch.cuda.synchronize()
    mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000)
    mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, 1)
    O, L = attend(h, m, q, starts, 512)
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_TIMEOUT
    none = torch.ones(tokens, dtype=torch.bool)
    none[starts[0]:starts[-1]] = False
    assert (O[none] == 7).all() and (L[none] == 7).all()
    mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, 0)
    mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
    O, L = attend(h, m, q, starts, 512)
    check(m, q, starts, O, L, [-1] * starts[0] + [0] * (starts[1] - starts[0]) + [1] * (starts[2] - starts[1]) + [-1] * (tokens - starts[2]))
    assert mx.mxgemm_get_device_status(h) == (0, 0)


def test_append_leaves_out_the_same_rows(h):
    """Rows before the first and behind the last sequence's are not appended."""
    m = Made([40, 20], 1, 64, 16)
    cache, table, lens = m.cache(), m.table_tensor(), torch.tensor(m.kv_len, dtype=torch.int32, device=DEV)
    new = torch.randn(12, 1, 64, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    mx.mxgemm_cache_append(h, cache, table, lens, new, -new, q_start=torch.tensor([5, 7, 10], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    got = [t.cpu() for t in m.dev]
    cache = m.cache()
    part = new[5:10].contiguous()
    mx.mxgemm_cache_append(h, cache, table, lens, part, -part, q_start=torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b.cpu()) for a, b in zip(got, m.dev))
