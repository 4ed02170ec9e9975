"""The 8-bit key/value cache on the GPU: append and attention against plain
64-bit implementations.

Append: every step of its definition is exact or one rounding to E4M3 (the
scales are powers of two), so codes and scales are equal.

Attention, per element of O: 2^-8 |O| for its rounding to BF16, and 2^-10 sum p|v|
for the weights: rounded to FP16 they are off by 2^-11 of themselves, the
logits (FP32 sums of exact products) by 2^-20 of sum |scale q k|, which the
inputs here keep under 64, so that exp is off by 2^-14.  lse: 2^-19 of
(1 + sum |scale q k|), twice the logits' error."""
import math

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def h():
    h = mx.mxgemm_create(0)
    yield h
    mx.mxgemm_destroy(h)


class Made:
    """A cache, a page table and lengths on the host; garbage (NaN codes) in all
    places that no sequence holds."""

    def __init__(self, kv_len, kv, d, page, seed=0, spare=3, extra=2, scales=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.kv_len, self.kv, self.d, self.page = list(kv_len), kv, d, page
        counts = [-(-t // page) for t in kv_len]
        self.pages = sum(counts) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = []
        for c in counts:
            self.table.append([order.pop() for _ in range(c)])
        self.width = max(counts + [1]) + extra
        codes = []
        for _ in range(2):
            c = (torch.randn(self.pages, kv, page, d, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            used = torch.zeros(self.pages, page, dtype=torch.bool)
            for row, t in zip(self.table, kv_len):
                for i, p in enumerate(row):
                    used[p, :max(0, min(page, t - i * page))] = True
            codes.append(torch.where(used[:, None, :, None], c, torch.tensor(0x7F, dtype=torch.uint8)))
        self.K, self.V = codes
        low, high = scales or (-9, -6)
        self.sK = torch.exp2(torch.randint(low, high, (self.pages, kv), generator=g).float())
        self.sV = torch.exp2(torch.randint(low, high, (self.pages, kv), generator=g).float()) * 1.37

    def table_tensor(self):
        t = torch.full((len(self.table), self.width), -7, dtype=torch.int32)
        for i, row in enumerate(self.table):
            t[i, :len(row)] = torch.tensor(row, dtype=torch.int32)
        return t.to(DEV)

    def cache(self):
        self.dev = [t.to(DEV) for t in (self.K, self.V, self.sK, self.sV)]
        return mx.Cache(*self.dev)


def starts_of(news):
    s = [0]
    for n in news:
        s.append(s[-1] + n)
    return s


def attend(h, m, q, news, scale=None, stream=None, lse=True, **kw):
    tokens, heads, _ = q.shape
    cache, table = m.cache(), m.table_tensor()
    lens = torch.tensor(m.kv_len, dtype=torch.int32, device=DEV)
    starts = None if news is None else torch.tensor(starts_of(news), dtype=torch.int32, device=DEV)
    O = torch.full((tokens, heads, m.d), math.nan, dtype=torch.bfloat16, device=DEV)
    L = torch.full((tokens, heads), math.nan, device=DEV) if lse else None
    mx.mxgemm_cache_attention(h, cache, table, lens, q if q.is_cuda else q.to(DEV), O, q_start=starts, scale=scale, lse=L, stream=stream, **kw)
    torch.cuda.synchronize()
    return O.cpu(), None if L is None else L.cpu()


def check(m, q, news, O, L, scale=None, **kw):
    scale = m.d ** -0.5 if scale is None else scale
    o, lse, mag, size = plain64.attention(plain64.value(m.K), m.sK, plain64.value(m.V), m.sV, m.table, m.kv_len, starts_of(news),
                                          q.cpu(), scale, **kw)
    assert float(size.max()) < 64 if size.numel() else True
    err, tol = (O.double() - o).abs(), 2.0 ** -8 * o.abs() + 2.0 ** -10 * mag
    assert not torch.isnan(O).any()
    assert (err <= tol).all(), f"O: worst {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"
    if L is not None:
        none = lse == -math.inf
        assert torch.equal(L == -math.inf, none) and (O[none] == 0).all()
        err = (L.double() - lse)[~none].abs()
        assert (err <= 2.0 ** -19 * (1 + size[~none])).all(), f"lse: worst {float(err.max())}"


def queries(m, tokens, heads, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, heads, m.d, generator=g) * 0.5).bfloat16()


DECODE = [  # lengths, kv heads, heads of a group, d, page
    ([1], 1, 1, 128, 16), ([0, 1, 2], 2, 4, 64, 16), ([15, 16, 17, 31, 32, 33], 1, 8, 128, 16), ([63, 64, 65, 127, 129], 2, 7, 128, 64),
    ([5, 300, 1], 3, 16, 64, 32), ([1000, 0, 77], 1, 5, 128, 128), ([2500], 2, 8, 128, 64), ([4097, 3], 1, 1, 128, 16), ([700] * 9, 1, 40, 64, 128),
]


@pytest.mark.parametrize("lens,kv,group,d,page", DECODE)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 4), (130, 17)])
def test_single_tokens(h, lens, kv, group, d, page, window, sinks):
    m = Made(lens, kv, d, page, seed=sum(lens))
    q = queries(m, len(lens), kv * group)
    O, L = attend(h, m, q, None, window=window, sinks=sinks)
    check(m, q, [1] * len(lens), O, L, window=window, sinks=sinks)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


PROMPT = [  # lengths, new tokens, kv heads, group, d, page
    ([5], [5], 1, 1, 128, 16), ([40, 3, 100], [2, 3, 0], 2, 4, 64, 32), ([300, 129], [130, 129], 1, 8, 128, 64),
    ([257, 64, 500], [1, 64, 333], 1, 2, 128, 128), ([0, 9], [0, 4], 1, 16, 64, 16), ([600, 2], [3, 2], 2, 7, 128, 16),
    ([1100], [1100], 1, 1, 128, 64), ([700, 701], [290, 17], 1, 3, 64, 64),
]


@pytest.mark.parametrize("lens,news,kv,group,d,page", PROMPT)
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 33, 5), (True, 1, 0), (False, 50, 2)])
def test_several_tokens(h, lens, news, kv, group, d, page, causal, window, sinks):
    m = Made(lens, kv, d, page, seed=sum(lens))
    q = queries(m, sum(news), kv * group)
    O, L = attend(h, m, q, news, causal=causal, window=window, sinks=sinks)
    check(m, q, news, O, L, causal=causal, window=window, sinks=sinks)


PROMPTS = [  # as PROMPT, with rows enough for whole tiles of the tensor cores
    ([300, 129], [130, 129], 8, 8, 128, 64), ([1100], [1100], 4, 4, 128, 64), ([257, 700, 500], [129, 300, 333], 6, 2, 64, 16),
    ([900, 64, 2], [300, 64, 2], 8, 7, 128, 32), ([513, 512, 511], [513, 200, 511], 8, 1, 128, 128), ([400], [257], 16, 3, 64, 128),
    ([0, 1500, 40], [9, 700, 31], 8, 4, 128, 16),
    # few row tiles: their keys are cut into parts
    ([5000], [70], 1, 1, 128, 64), ([3001, 0, 129], [40, 2, 100], 1, 8, 64, 32), ([2500, 2600], [64, 1], 2, 4, 128, 128),
]


@pytest.mark.parametrize("lens,news,kv,group,d,page", PROMPTS)
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 33, 5), (True, 200, 130), (False, 50, 2)])
def test_prompts(h, lens, news, kv, group, d, page, causal, window, sinks):
    m = Made(lens, kv, d, page, seed=sum(lens))
    q = queries(m, sum(news), kv * group)
    O, L = attend(h, m, q, news, causal=causal, window=window, sinks=sinks)
    check(m, q, news, O, L, causal=causal, window=window, sinks=sinks)
    again, L2 = attend(h, m, q, news, causal=causal, window=window, sinks=sinks)
    assert torch.equal(O, again) and torch.equal(L, L2)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


@pytest.mark.parametrize("lens,news,kv,d", [([2500], [64], 160, 64), ([1900, 700, 64], [70, 64, 66], 60, 128),
                                             ([40, 2000], [40, 300], 80, 64)])
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 700, 130)])
def test_prompts_of_more_row_tiles_than_sms(h, lens, news, kv, d, causal, window, sinks):
    """The row tiles past a multiple of the SMs have their keys cut for several CTAs."""
    m = Made(lens, kv, d, 16, seed=kv)
    q = queries(m, sum(news), kv)
    O, L = attend(h, m, q, news, causal=causal, window=window, sinks=sinks)
    check(m, q, news, O, L, causal=causal, window=window, sinks=sinks)
    again, L2 = attend(h, m, q, news, causal=causal, window=window, sinks=sinks)
    assert torch.equal(O, again) and torch.equal(L, L2)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


@pytest.mark.parametrize("f,scale", [(2.0 ** 20, 0.08), (2.0 ** -40, 0.08), (1.0, -0.1)])
def test_prompts_with_wide_scales(h, f, scale):
    """Page scales over 2^30, queries past FP16's range, a negative scale."""
    m = Made([300, 250], 8, 128, 16, scales=(-30, 0))
    m.sK.fill_(2.0 ** -8)
    m.table[0][3], m.table[1][0] = -1, m.pages
    q = (queries(m, 300, 32).float() * f).bfloat16()
    O, L = attend(h, m, q, [200, 100], scale=scale / f)
    check(m, q, [200, 100], O, L, scale=scale / f)
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_INVALID_VALUE


def test_long_sequence_is_split(h):
    m = Made([20011, 64], 1, 128, 64)
    q = queries(m, 2, 8)
    O, L = attend(h, m, q, None)
    check(m, q, [1, 1], O, L)
    again, L2 = attend(h, m, q, None)
    assert torch.equal(O, again) and torch.equal(L, L2)


@pytest.mark.parametrize("n,kv,group,d,page", [(40, 4, 4, 128, 32), (50, 2, 8, 64, 16), (33, 3, 2, 64, 128), (130, 1, 16, 128, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_many_sequences(h, n, kv, group, d, page, window, sinks):
    """More sequences than a warp counts at a time, and more heads of theirs than
    CTAs are handed out for one by one; every seventh or so is empty."""
    lens = [37 * i * i % 701 * (i % 7 != 3) for i in range(n)]
    m = Made(lens, kv, d, page, seed=n)
    q = queries(m, n, kv * group)
    O, L = attend(h, m, q, None, window=window, sinks=sinks)
    check(m, q, [1] * n, O, L, window=window, sinks=sinks)
    again, L2 = attend(h, m, q, None, window=window, sinks=sinks)
    assert torch.equal(O, again) and torch.equal(L, L2)


def test_queries_before_the_first_key(h):
    """More queries than the sequence has tokens: the first ones see nothing."""
    m = Made([3, 0, 200], 1, 64, 16)
    news = [7, 2, 1]
    q = queries(m, 10, 2)
    O, L = attend(h, m, q, news)
    check(m, q, news, O, L)
    assert (L[:4] == -math.inf).all() and (O[:4] == 0).all()


@pytest.mark.parametrize("news", [None, [70, 100]])
def test_scales_that_differ_by_page(h, news):
    """Page scales over a range of 2^30: the weights keep their precision where
    the keys that count most stand in pages of small values."""
    m = Made([180, 250], 2, 128, 16, scales=(-30, 0))
    m.sK.fill_(2.0 ** -8)
    q = queries(m, 2 if news is None else 170, 8)
    O, L = attend(h, m, q, news)
    check(m, q, news or [1, 1], O, L)


def test_large_and_tiny_queries(h):
    """Queries past FP16's range, with the scale that makes their logits ordinary."""
    m = Made([100, 90], 1, 128, 32)
    for f in (2.0 ** 20, 2.0 ** -40):
        q = (queries(m, 2, 4).float() * f).bfloat16()
        O, L = attend(h, m, q, None, scale=0.08 / f)
        check(m, q, [1, 1], O, L, scale=0.08 / f)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    O, L = attend(h, m, q, None)
    check(m, q, [1, 1], O, L)


@pytest.mark.parametrize("news", [None, [40, 200]])
def test_negative_scale_and_no_lse(h, news):
    m = Made([100, 300], 1, 64, 32)
    q = queries(m, 2 if news is None else 240, 4)
    O, _ = attend(h, m, q, news, scale=-0.1, lse=False)
    check(m, q, news or [1, 1], O, None, scale=-0.1)


@pytest.mark.parametrize("news", [None, [1, 150]])
def test_strided_queries_and_other_stream(h, news):
    m = Made([100, 300], 2, 64, 32)
    n = 2 if news is None else 151
    wide = queries(m, n, 12).to(DEV)
    q = wide[:, 4:8]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        O, L = attend(h, m, q, news, stream=s)
    check(m, q, news or [1, 1], O, L)


@pytest.mark.parametrize("news", [None, [130, 3]])
def test_page_numbers_that_name_no_page(h, news):
    m = Made([150, 50], 1, 64, 16)
    m.table[0][3], m.table[0][9], m.table[1][0] = -1, m.pages, 2 ** 31 - 1
    q = queries(m, 2 if news is None else 133, 4)
    O, L = attend(h, m, q, news)
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_INVALID_VALUE
    check(m, q, news or [1, 1], O, L)
    assert mx.mxgemm_get_device_status(h) == (0, 0)


def test_lengths_that_do_not_fit(h):
    m = Made([40, 50], 1, 64, 16)
    q = queries(m, 2, 4)
    real, m.kv_len = m.kv_len, [10 ** 9, 50]
    O, L = attend(h, m, q, None)
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_INVALID_VALUE
    m.kv_len = [0, 50]
    check(m, q, [1, 1], O, L)
    m.kv_len = [-3, 50]
    O, L = attend(h, m, q, None)
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_INVALID_VALUE
    m.kv_len = [0, 50]
    check(m, q, [1, 1], O, L)


def do_append(h, m, x, y, news, stream=None):
    cache, table = m.cache(), m.table_tensor()
    lens = torch.tensor(m.kv_len, dtype=torch.int32, device=DEV)
    starts = None if news is None else torch.tensor(starts_of(news), dtype=torch.int32, device=DEV)
    mx.mxgemm_cache_append(h, cache, table, lens, x, y, q_start=starts, stream=stream)
    torch.cuda.synchronize()
    return [t.cpu() for t in m.dev]


APPEND = [  # lengths with the new tokens, new tokens (None: one each), kv heads, d, page
    ([1, 16, 17, 33], None, 2, 64, 16), ([100, 1, 64, 65], None, 1, 128, 64), ([5, 130, 0, 77], [5, 100, 0, 1], 2, 64, 32),
    ([500], [500], 3, 128, 128), ([300, 301, 302], [17, 300, 111], 1, 128, 16), ([1000, 128], [999, 128], 1, 64, 64), ([200] * 40, None, 1, 64, 128),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-3, 1.0, 100.0])
@pytest.mark.parametrize("lens,news,kv,d,page", APPEND)
def test_append(h, lens, news, kv, d, page, size, dtype):
    m = Made(lens, kv, d, page, seed=sum(lens))
    m.sV.copy_(m.sK)
    n = news or [1] * len(lens)
    wide = (torch.randn(sum(n), 4 * kv, d, generator=m.g) * size * torch.exp(torch.randn(sum(n), 1, 1, generator=m.g))).to(dtype)
    wide[::3, kv:2 * kv] = 0
    wide = wide.to(DEV)
    x, y = wide[:, kv:2 * kv], wide[:, 3 * kv:]
    K, V, sK, sV = do_append(h, m, x, y, news)
    for codes, scale, old, olds, new in ((K, sK, m.K, m.sK, x), (V, sV, m.V, m.sV, y)):
        want, ws = plain64.value(old), olds.double()
        plain64.append(want, ws, m.table, lens, starts_of(n), new.cpu())
        assert torch.equal(scale.double(), ws)
        got = plain64.value(codes)
        assert torch.equal(torch.nan_to_num(got, nan=999.0), torch.nan_to_num(want, nan=999.0))
    assert mx.mxgemm_get_device_status(h) == (0, 0)


def test_token_by_token_is_the_prompt_where_scales_do_not_grow(h):
    """Tokens of one size appended one by one: the codes of one append of all."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(70, 1, 64, generator=g).clamp(-3.4, 3.4)
    x[:, :, 0] = 3.5  # every token needs the same scale
    m = Made([70], 1, 64, 32)
    whole = do_append(h, m, x.to(DEV), x.to(DEV), [70])
    for t in range(70):
        m.kv_len = [t + 1]
        m.K, m.V, m.sK, m.sV = do_append(h, m, x[t:t + 1].to(DEV), x[t:t + 1].to(DEV), None)
    for a, b in zip(whole, (m.K, m.V, m.sK, m.sV)):
        assert torch.equal(a, b)


def test_append_leaves_bad_sequences_alone(h):
    m = Made([40, 50, 20], 1, 64, 16)
    m.table[0][2] = -1
    x = torch.randn(3, 1, 64, generator=m.g).to(DEV)
    m.kv_len = [40, 10 ** 9, 0]  # an absent page, a length past the table, a length shorter than its new tokens
    K, V, sK, sV = do_append(h, m, x, x, None)
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_INVALID_VALUE
    assert torch.equal(K, m.K) and torch.equal(V, m.V) and torch.equal(sK, m.sK) and torch.equal(sV, m.sV)


def test_cache_past_32_bits(h):
    """Pages whose codes lie past 2^32 bytes of K and V."""
    pages, page, d = 270000, 128, 128
    K = torch.zeros(pages, 1, page, d, dtype=torch.uint8, device=DEV)
    V, s = torch.zeros_like(K), torch.ones(pages, 1, device=DEV)
    cache = mx.Cache(K, V, s, s.clone())
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device=DEV)
    n = 300
    g = torch.Generator().manual_seed(5)
    x = torch.randn(n, 2, d, generator=g).bfloat16()
    lens, starts = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
    xd = x.to(DEV)
    mx.mxgemm_cache_append(h, cache, table, lens, xd[:, :1], xd[:, 1:], q_start=starts)
    at = [pages - 1, 3, pages - 2]
    m = Made([n], 1, d, page, spare=0)
    m.table = [[0, 1, 2]]
    m.K, m.V, m.sK, m.sV = (t[at].cpu() for t in (K, V, cache.K_scale, cache.V_scale))
    for codes, scale, new in ((m.K, m.sK, x[:, :1]), (m.V, m.sV, x[:, 1:])):
        want, ws = torch.zeros(codes.shape, dtype=torch.float64), torch.ones(3, 1, dtype=torch.float64)
        plain64.append(want, ws, m.table, [n], [0, n], new)
        assert torch.equal(scale.double(), ws) and torch.equal(plain64.value(codes), want)
    assert int(K.count_nonzero()) == int(m.K.count_nonzero())
    q = queries(m, 5, 4)
    O = torch.empty(5, 4, d, dtype=torch.bfloat16, device=DEV)
    L = torch.empty(5, 4, device=DEV)
    mx.mxgemm_cache_attention(h, cache, table, lens, q.to(DEV), O, q_start=torch.tensor([0, 5], dtype=torch.int32, device=DEV), lse=L)
    check(m, q, [5], O.cpu(), L.cpu())


def test_refusals(h):
    m = Made([40], 2, 64, 16)
    cache, table = m.cache(), m.table_tensor()
    lens = torch.tensor([40], dtype=torch.int32, device=DEV)
    q = queries(m, 1, 4).to(DEV)
    O = torch.empty_like(q)
    x = torch.zeros(1, 2, 64, device=DEV)
    att = lambda hh=h, c=cache, t=table, le=lens, qq=q, o=O, **kw: mx.mxgemm_cache_attention(hh, c, t, le, qq, o, check=False, **kw)
    app = lambda hh=h, c=cache, a=x, b=x, **kw: mx.mxgemm_cache_append(hh, c, table, lens, a, b, check=False, **kw)
    assert att() == mx.OK and app() == mx.OK
    assert att(hh=None) == mx.ERR_INVALID_VALUE and app(hh=None) == mx.ERR_INVALID_VALUE
    for bad in (dict(scale=math.inf), dict(scale=math.nan), dict(window=-1), dict(sinks=-1), dict(le=lens.cpu()), dict(t=table.cpu()), dict(qq=q.cpu()),
                dict(qq=queries(m, 1, 3).to(DEV), o=torch.empty(1, 3, 64, dtype=torch.bfloat16, device=DEV))):
        assert att(**bad) == mx.ERR_INVALID_VALUE, bad
    wide = torch.zeros(200, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert att(qq=wide.view(-1)[4:260].view(1, 4, 64)) == mx.ERR_MISALIGNED
    assert app(a=x.cpu(), b=x.cpu()) == mx.ERR_INVALID_VALUE
    f = torch.zeros(400, device=DEV)
    assert app(a=f[1:129].view(1, 2, 64), b=f[1:129].view(1, 2, 64)) == mx.ERR_MISALIGNED
    for shape in ((3, 2, 24, 64), (3, 2, 16, 96)):
        c = mx.Cache(*(torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2)), *(torch.ones(shape[:2], device=DEV) for _ in range(2)))
        d = shape[3]
        qq = torch.zeros(1, 4, d, dtype=torch.bfloat16, device=DEV)
        assert att(c=c, qq=qq, o=torch.empty_like(qq)) == mx.ERR_INVALID_VALUE
    for call in (lambda: att(qq=q.float()), lambda: att(o=O.float()), lambda: att(lse=torch.empty(2, 4, device=DEV)), lambda: att(le=lens.float()),
                 lambda: att(t=table.long()), lambda: att(q_start=lens), lambda: app(a=x.half(), b=x.half()), lambda: app(b=x[:, :1]),
                 lambda: mx.Cache(m.K, m.V, m.sK[:1], m.sV), lambda: mx.Cache(m.K.float(), m.V.float(), m.sK, m.sV)):
        with pytest.raises(ValueError):
            call()


def test_nothing_to_do(h):
    m = Made([0], 1, 64, 16)
    cache, table = m.cache(), m.table_tensor()
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    starts = torch.zeros(2, dtype=torch.int32, device=DEV)
    mx.mxgemm_cache_attention(h, cache, table, lens, none, none.clone(), q_start=starts)
    mx.mxgemm_cache_append(h, cache, table, lens, none[:, :1], none[:, :1].clone(), q_start=starts)
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    mx.mxgemm_cache_attention(h, cache, table[:0], empty, none, none.clone())


def test_layer_example():
    """The example layer (quantizer, products, append and attention together),
    prompt and single tokens, against FP32.  E4M3 rounds each value by 2^-4 of
    itself at most, 0.027 of it in root mean square (uniform over a binade's
    steps); the layer rounds x, two weights, K or V, and o, five times, their
    errors independent: under 0.07 of the output's norm, twice that allowed."""
    import importlib.util
    from pathlib import Path
    path = Path(__file__).resolve().parents[1] / "examples" / "attention_layer_8bit.py"
    spec = importlib.util.spec_from_file_location("attention_layer_8bit", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    error, _ = example.run(batch=3, prompt=333, steps=3, model=512, heads=8, kv_heads=2, d=64, page=32)
    assert error < 0.14
    error, _ = example.run(batch=2, prompt=300, steps=2, model=1024, heads=16, kv_heads=8, d=128, page=64)
    assert error < 0.14


def test_captured_in_a_graph(h):
    """A decoding step captured once and replayed with longer sequences."""
    m = Made([70, 40, 9], 2, 128, 32)
    cache, table = m.cache(), m.table_tensor()
    lens = torch.tensor([60, 30, 5], dtype=torch.int32, device=DEV)
    q, x = queries(m, 3, 8).to(DEV), torch.randn(3, 2, 128, generator=m.g).to(DEV)
    O = torch.empty_like(q)

    def step():
        s = torch.cuda.current_stream()
        mx.mxgemm_cache_append(h, cache, table, lens, x, x, stream=s)
        mx.mxgemm_cache_attention(h, cache, table, lens, q, O, stream=s)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens += 1
    x.normal_()
    step()
    want, kept = O.clone(), [t.clone() for t in m.dev]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, want) and all(torch.equal(a, b) for a, b in zip(m.dev, kept))
