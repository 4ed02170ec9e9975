"""The product with a scale for each block of 128 and its quantizer on the GPU,
against plain 64-bit implementations.

Tolerance of a product, per element: FP32 output 1e-5 * sum |terms| (the rule
of the other products here): the tensor cores' sum of a block is off by a few
2^-23 of its terms, the scaling by two roundings and the sum of ceil(K/128)
blocks by as many, 2^-24 each: under 5e-6 for K <= 8192.  BF16 output adds its
rounding, 2^-8 |C|.  Small integers with powers of two as scales are exact.
The quantizer's FP32 steps are fixed by its definition: equal bits."""
import math

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def handles():
    hs = {}
    for nk in (True, False):
        h = mx.mxgemm_create(0)
        mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K if nk else mx.B_K_BY_N)
        hs[nk] = h
    yield hs
    for h in hs.values():
        mx.mxgemm_destroy(h)


def random_codes(shape, g):
    c = torch.randint(0, 254, shape, generator=g)
    return torch.where(c >= 127, c + 1, c).to(torch.uint8)  # no NaN codes


def operands(m, n, k, b_block, seed, codes=random_codes):
    g = torch.Generator().manual_seed(seed)
    kb = -(-k // 128)
    a, b = codes((m, k), g), codes((n, k), g)
    sa = torch.exp(torch.randn(m, kb, generator=g))
    sb = torch.exp(torch.randn(n if b_block == 1 else -(-n // 128), kb, generator=g))
    return a, sa, b, sb


def run(h, nk, a, sa, b, sb, b_block, out="f32", c=None, stream=None):
    m, k = a.shape
    n = b.shape[0]
    if not nk:
        b, sb = b.t().contiguous(), sb.t().contiguous()
    a, sa, b, sb = (t.to(DEV) for t in (a, sa, b, sb))
    dt = torch.float32 if out == "f32" else torch.bfloat16
    C = torch.full((m, n), math.nan, dtype=dt, device=DEV) if c is None else c.to(DEV, dt)
    mx.mxgemm_run_block128(h, m, n, k, a, sa, b, sb, C, use_acc=c is not None,
                           out_dtype=mx.OUT_F32 if out == "f32" else mx.OUT_BF16, b_block=b_block, stream=stream)
    torch.cuda.synchronize()
    assert mx.mxgemm_get_device_status(h) == (0, 0)
    return C.cpu()


def check(C, ref, mag, out):
    tol = 1e-5 * mag + (2.0 ** -8 * ref.abs() if out == "bf16" else 0)
    err = (C.double() - ref).abs()
    assert torch.isfinite(C).all()
    assert (err <= tol).all(), f"worst {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"


SHAPES = [  # m, n, k: tiles not full, blocks not full, one row, one column, K of one partial block
    (1, 1, 16), (1, 128, 128), (1, 257, 400), (7, 100, 2048), (16, 1000, 1040), (33, 500, 512), (64, 384, 96),
    (100, 256, 144), (128, 128, 4096), (129, 257, 272), (200, 1, 640), (256, 256, 128), (300, 520, 1168),
    (513, 777, 384), (700, 300, 4112), (130, 2000, 8192),
]


@pytest.mark.parametrize("b_block", [128, 1])
@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(handles, m, n, k, nk, b_block):
    n = n if nk else -(-n // 16) * 16
    a, sa, b, sb = operands(m, n, k, b_block, m * 7 + n + k)
    ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, b_block)
    for out in ("f32", "bf16"):
        check(run(handles[nk], nk, a, sa, b, sb, b_block, out), ref, mag, out)


@pytest.mark.parametrize("b_block", [128, 1])
def test_whole_and_split_tiles_together(handles, b_block):
    """99 tiles: a full wave of whole ones, and 23 whose K is split over the idle
    pairs, added in a fixed order."""
    m, n, k = 2600, 2300, 4096
    a, sa, b, sb = operands(m, n, k, b_block, 12)
    ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, b_block)
    C = run(handles[True], True, a, sa, b, sb, b_block)
    check(C, ref, mag, "f32")
    assert torch.equal(C, run(handles[True], True, a, sa, b, sb, b_block))


@pytest.mark.parametrize("m,n,k", [(5, 300, 272), (300, 300, 272), (300, 257, 4096)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_accumulates(handles, m, n, k, out):
    a, sa, b, sb = operands(m, n, k, 128, 5)
    c = torch.randn(m, n, generator=torch.Generator().manual_seed(9)) * 1000
    c = c if out == "f32" else c.bfloat16()
    ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, 128)
    check(run(handles[True], True, a, sa, b, sb, 128, out, c), ref + c.double(), mag + c.double().abs(), out)


@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("m,n,k", [(3, 272, 1024), (40, 272, 1024), (300, 272, 1024), (520, 512, 400)])
def test_exact_integers_and_block_places(handles, m, n, k, nk):
    """Integers up to 8 and scales that are powers of two, another for each
    block: every sum is exact, so one scale read from a wrong place shows."""
    ints = torch.tensor([0x00, 0x38, 0x40, 0x44, 0x48, 0x4A, 0x4C, 0x4E, 0x50], dtype=torch.uint8)
    codes = lambda shape, g: ints[torch.randint(0, 9, shape, generator=g)] | (torch.randint(0, 2, shape, generator=g) << 7).to(torch.uint8)
    for b_block in (128, 1):
        a, sa, b, sb = operands(m, n, k, b_block, 3, codes)
        g = torch.Generator().manual_seed(4)
        sa = torch.exp2(torch.randint(-2, 3, sa.shape, generator=g).float())
        sb = torch.exp2(torch.randint(-2, 3, sb.shape, generator=g).float())
        ref, _ = plain64.product(plain64.value(a), sa, plain64.value(b), sb, b_block)
        assert torch.equal(run(handles[nk], nk, a, sa, b, sb, b_block).double(), ref)


@pytest.mark.parametrize("m", [20, 300])
@pytest.mark.parametrize("fa,fb", [(1, 0), (0, 1), (1, 1)])
def test_e5m2_operands(m, fa, fb):
    g = torch.Generator().manual_seed(1)
    codes = lambda shape, g: (torch.randint(0, 0x7C, shape, generator=g) | (torch.randint(0, 2, shape, generator=g) << 7)).to(torch.uint8)
    a, sa, b, sb = operands(m, 300, 272, 128, 2, codes)
    a = a if fa else random_codes(a.shape, g)
    b = b if fb else random_codes(b.shape, g)
    h = mx.mxgemm_create(0)
    try:
        mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
        mx.mxgemm_set_option(h, mx.OPT_A_FORMAT, mx.FMT_E5M2 if fa else mx.FMT_E4M3)
        mx.mxgemm_set_option(h, mx.OPT_B_FORMAT, mx.FMT_E5M2 if fb else mx.FMT_E4M3)
        val = lambda c, f: plain64.value_e5m2(c) if f else plain64.value(c)
        ref, mag = plain64.product(val(a, fa), sa, val(b, fb), sb, 128)
        check(run(h, True, a, sa, b, sb, 128), ref, mag, "f32")
    finally:
        mx.mxgemm_destroy(h)


@pytest.mark.parametrize("m", [8, 300])
def test_nan_stays_in_its_row_and_column(handles, m):
    a, sa, b, sb = operands(m, 300, 528, 128, 8)
    a[3, 500] = 0x7F
    b[270, 17] = 0xFF
    C = run(handles[True], True, a, sa, b, sb, 128)
    nan = torch.isnan(C)
    want = torch.zeros_like(nan)
    want[3], want[:, 270] = True, True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("m", [16, 400])
def test_other_stream_and_equal_bits(handles, m):
    a, sa, b, sb = operands(m, 640, 2064, 128, 6)
    first = run(handles[True], True, a, sa, b, sb, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run(handles[True], True, a, sa, b, sb, 128, stream=s)
    assert torch.equal(first, again)


def test_nothing_past_the_result(handles):
    """Rows and columns past C's edge are not written: C inside a guarded buffer."""
    for m, n in ((5, 37), (300, 301)):
        a, sa, b, sb = operands(m, n, 272, 128, 11)
        buf = torch.full((m * n + 64,), 7.5, device=DEV)
        C = buf[:m * n]
        d = [t.to(DEV) for t in (a, sa, b, sb)]
        mx.mxgemm_run_block128(handles[True], m, n, 272, *d, C, stream=None)
        torch.cuda.synchronize()
        assert (buf[m * n:] == 7.5).all()
        ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, 128)
        check(C.view(m, n).cpu(), ref, mag, "f32")


def test_product_refusals(handles):
    t = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    f = torch.zeros(1 << 12, device=DEV)
    ok = dict(h=handles[True], M=32, N=32, K=32, A=t, A_scale=f, B=t, B_scale=f, C=f, check=False)
    call = lambda **kw: mx.mxgemm_run_block128(**{**ok, **kw})
    assert call() == mx.OK
    assert call(M=0) == mx.OK and call(N=0) == mx.OK
    for bad in (dict(M=-1), dict(K=24), dict(K=1 << 31), dict(b_block=64), dict(out_dtype=2), dict(A=None),
                dict(A_scale=None), dict(B=None), dict(B_scale=None), dict(C=None), dict(C=torch.zeros(9)),
                dict(A=torch.zeros(64, dtype=torch.uint8)), dict(h=None), dict(h=handles[False], N=24)):
        assert call(**bad) == mx.ERR_INVALID_VALUE, bad
    for bad in (dict(A=t[8:]), dict(B=t[8:]), dict(C=f[1:]), dict(A_scale=t[2:])):
        assert call(**bad) == mx.ERR_MISALIGNED, bad
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_A_FORMAT, mx.FMT_E2M1)
    assert call(h=h) == mx.ERR_INVALID_VALUE
    mx.mxgemm_destroy(h)


def test_no_contraction(handles):
    c = torch.full((4, 8), 3.0, device=DEV)
    mx.mxgemm_run_block128(handles[True], 4, 8, 0, None, None, None, None, c, use_acc=1)
    assert (c == 3).all()
    mx.mxgemm_run_block128(handles[True], 4, 8, 0, None, None, None, None, c)
    assert (c == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block", ["rows", "cols", "tiles"])
@pytest.mark.parametrize("r,c", [(1, 16), (1, 4096), (3, 144), (127, 128), (128, 256), (130, 272), (257, 1040), (1000, 2048)])
def test_quantizer(r, c, block, dtype):
    g = torch.Generator().manual_seed(r + c)
    x = torch.randn(r, c, generator=g) * torch.exp(2 * torch.randn(r, 1, generator=g))
    x[:, ::7] *= 50
    x[r // 2, : c // 2] = 0
    if r > 128:
        x[128:] = 0  # blocks of zeros
    x[0, 0] = 1e-35  # far below its block's largest
    x = x.to(dtype)
    want, scales = plain64.quantize(x, block)
    codes = torch.full(want.shape, 0x55, dtype=torch.uint8, device=DEV)
    sc = torch.full(scales.shape, math.nan, device=DEV)
    mx.mxgemm_quantize_block128(x.to(DEV), r, c, codes, sc,
                                block={"rows": mx.BLOCK_ROWS, "cols": mx.BLOCK_COLS, "tiles": mx.BLOCK_TILES}[block])
    torch.cuda.synchronize()
    assert torch.equal(sc.cpu(), scales.contiguous())
    assert torch.equal(plain64.value(codes.cpu()), want)


def test_quantizer_extremes():
    """Largest and smallest finite values; a block whose largest is subnormal."""
    x = torch.tensor([[3.4e38, -3.4e38, 1.0, 1e-38] + [0.0] * 124, [1e-40, -1e-44] + [0.0] * 126])
    want, scales = plain64.quantize(x, "rows")
    codes = torch.empty(2, 128, dtype=torch.uint8, device=DEV)
    sc = torch.empty(2, 1, device=DEV)
    mx.mxgemm_quantize_block128(x.to(DEV), 2, 128, codes, sc)
    assert torch.equal(sc.cpu(), scales) and torch.equal(plain64.value(codes.cpu()), want)


def test_quantizer_refusals():
    x, c, s = torch.zeros(64, 64, device=DEV), torch.zeros(4096, dtype=torch.uint8, device=DEV), torch.zeros(64, device=DEV)
    call = lambda X=x, R=64, C=64, codes=c, scales=s, **kw: mx.mxgemm_quantize_block128(X, R, C, codes, scales, check=False, **kw)
    assert call() == mx.OK and call(R=0) == mx.OK
    for bad in (dict(C=24), dict(R=-1), dict(block=3), dict(x_dtype=2), dict(X=None, x_dtype=0), dict(codes=None), dict(scales=None),
                dict(X=torch.zeros(64, 64))):
        assert call(**bad) == mx.ERR_INVALID_VALUE, bad
    assert call(codes=c[8:]) == mx.ERR_MISALIGNED and call(X=x.view(-1)[1:]) == mx.ERR_MISALIGNED


def test_layer_forward_and_gradients(handles):
    """Y = X W^T, dX = dY W and dW = dY^T X through the quantizer and the three
    forms of the product, against the formulas on the quantized values; and the
    gradients against differences of the forward product in 64 bits."""
    g = torch.Generator().manual_seed(0)
    T, I, O = 300, 272, 400
    x, w, dy = torch.randn(T, I, generator=g), torch.randn(O, I, generator=g) * 0.05, torch.randn(T, O, generator=g)

    def quant(t, block):
        r, c = t.shape
        want, scales = plain64.quantize(t, block)
        codes = torch.empty(want.shape, dtype=torch.uint8, device=DEV)
        sc = torch.empty(scales.shape, device=DEV)
        mx.mxgemm_quantize_block128(t.to(DEV), r, c, codes, sc, block={"rows": 0, "cols": 1, "tiles": 2}[block])
        return codes, sc

    def prod(nk, a, b, n, b_block):
        (ca, sa), (cb, sb) = a, b
        C = torch.empty(ca.shape[0], n, device=DEV)
        mx.mxgemm_run_block128(handles[nk], ca.shape[0], n, ca.shape[1], ca, sa, cb, sb, C, b_block=b_block)
        return C.cpu().double()

    W = quant(w, "tiles")
    y = prod(True, quant(x, "rows"), W, O, 128)
    dx = prod(False, quant(dy, "rows"), W, I, 128)
    dw = prod(True, quant(dy, "cols"), quant(x, "cols"), I, 1)

    def deq(t, block):
        v, s = plain64.quantize(t, block)
        if block == "rows":
            return v * plain64.spread(s, 1, v.shape[1])
        if block == "cols":
            return (v * plain64.spread(s, 1, v.shape[1])).t()[:t.shape[0]]
        return v * plain64.spread(s, 0, v.shape[0]).repeat_interleave(128, 1)[:, :v.shape[1]]

    wq = deq(w, "tiles")
    for got, left, right in ((y, deq(x, "rows"), wq.t()), (dx, deq(dy, "rows"), wq), (dw, deq(dy, "cols").t(), deq(x, "cols"))):
        assert ((got - left @ right).abs() <= 1e-5 * (left.abs() @ right.abs())).all()
    # differences of L = sum(dY * (X W^T)), linear in X and in W: exact up to the quantization of dY, X and W,
    # 2^-4 of each value at most (E4M3 normals; smaller values 2^-10 of their block's largest)
    for (i, j) in ((0, 0), (17, 200), (299, 271)):
        diff = float((dy[i].double() * w[:, j].double()).sum())
        assert abs(float(dx[i, j]) - diff) <= float((0.14 * dy[i].abs() * w[:, j].abs()).sum()) + 0.01 * O * float(dy.abs().max() * w.abs().max())
    for (i, j) in ((0, 0), (399, 271)):
        diff = float((dy[:, i].double() * x[:, j].double()).sum())
        assert abs(float(dw[i, j]) - diff) <= float((0.14 * dy[:, i].abs() * x[:, j].abs()).sum()) + 0.01 * T * float(dy.abs().max() * x.abs().max())


def test_past_32_bits(handles):
    """C of more than 2^31 elements and more than 2^32 bytes: rows from its end."""
    m, n, k = 70000, 32768, 16
    g = torch.Generator().manual_seed(3)
    a, b = random_codes((m, k), g), random_codes((n, k), g)
    sa, sb = torch.rand(m, 1, generator=g) + 0.5, torch.rand(n // 128, 1, generator=g) + 0.5
    C = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    mx.mxgemm_run_block128(handles[True], m, n, k, a.to(DEV), sa.to(DEV), b.to(DEV), sb.to(DEV), C, out_dtype=mx.OUT_BF16)
    rows = torch.tensor([0, 65535, 65536, 69998, 69999])
    ref, mag = plain64.product(plain64.value(a[rows]), sa[rows], plain64.value(b), sb, 128)
    check(C[rows.to(DEV)].cpu(), ref, mag, "bf16")


@pytest.mark.parametrize("m,b_block", [(16, 128), (300, 128), (300, 1)])
def test_a_stalled_producer_ends_in_a_status(m, b_block):
    """No loads: every wait runs out, the kernel returns, the handle stays usable."""
    h = mx.mxgemm_create(0)
    try:
        mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
        a, sa, b, sb = operands(m, 300, 400, b_block, 1)
        dev = [t.to(DEV) for t in (a, sa, b, sb)]
        C = torch.zeros(m, 300, device=DEV)
        mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 50_000_000)
        mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, 1)
        mx.mxgemm_run_block128(h, m, 300, 400, *dev, C, b_block=b_block)
        assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_TIMEOUT
        mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, 0)
        mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
        ref, mag = plain64.product(plain64.value(a), sa, plain64.value(b), sb, b_block)
        check(run(h, True, a, sa, b, sb, b_block), ref, mag, "f32")
    finally:
        mx.mxgemm_destroy(h)


def test_profile_events_and_launch_count(handles):
    a, sa, b, sb = (t.to(DEV) for t in operands(40, 256, 256, 128, 1))
    C = torch.empty(40, 256, device=DEV)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ev:
        e.record()
    h = handles[True]
    n = mx.mxgemm_get_launch_count(h)
    mx.mxgemm_set_profile_events(h, *ev)
    try:
        mx.mxgemm_run_block128(h, 40, 256, 256, a, sa, b, sb, C)
    finally:
        mx.mxgemm_set_profile_events(h, None, None)
    torch.cuda.synchronize()
    assert mx.mxgemm_get_launch_count(h) == n + 1 and ev[0].elapsed_time(ev[1]) > 0


def test_captured_in_a_graph(handles):
    """The product and its quantizer hold no host state: captured once, replayed on new inputs."""
    T, I, O = 300, 272, 400
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn(T, I, generator=g).to(DEV), torch.randn(O, I, generator=g).to(DEV)
    xc, xs = torch.empty(T, I, dtype=torch.uint8, device=DEV), torch.empty(T, 3, device=DEV)
    wc, ws = torch.empty(O, I, dtype=torch.uint8, device=DEV), torch.empty(4, 3, device=DEV)
    C = torch.empty(T, O, device=DEV)

    def step():
        s = torch.cuda.current_stream()
        mx.mxgemm_quantize_block128(x, T, I, xc, xs, stream=s)
        mx.mxgemm_quantize_block128(w, O, I, wc, ws, block=mx.BLOCK_TILES, stream=s)
        mx.mxgemm_run_block128(handles[True], T, O, I, xc, xs, wc, ws, C, stream=s)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn(T, I, generator=g))
    step()
    want = C.clone()
    C.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, want)
