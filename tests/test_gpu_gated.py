"""The gated pair of products and its gradient on the GPU, against plain 64-bit
implementations.

Tolerance of g and u, per element: 1e-5 * sum |terms|, as for the single product
(tests/test_gpu_block128.py).  H = act(g) u moves by |act'| <= 1.13 times g's error
times |u|, and by |act| <= |g| times u's; the activation itself is off by 2^-20 of
its value at |x| <= 16 (ex2.approx 2^-22, its argument's rounding 2^-24 |x| 1.45, the
reciprocal 2^-23, and as many products), and past that by 2^-24 |x| more, which counts
where the logistic function is under e^-16 alone; so 2^-18 covers it to |x| = 80, below
which the value is under 2^-115 of its argument.  BF16 output adds 2^-8 of the value.
A code stands for its value to 2^-4 of it (half a step) or 2^-10 of the scale (half the
least step); a scale is the row's largest value / 448, off by as much as the values."""
import math

import pytest
import torch

import plain64

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"
ACTS = {"silu": 0, "gelu": 1}
CUBE = 0.044715


def act64(g, act):
    """The activation and its derivative: g times a logistic function in both (1 + tanh
    would lose small values even in 64 bits)."""
    c = 2 * math.sqrt(2 / math.pi)
    p, slope = (torch.sigmoid(g), 1.0) if act == "silu" else (torch.sigmoid(c * (g + CUBE * g ** 3)), c * (1 + 3 * CUBE * g ** 2))
    q = torch.sigmoid(-g) if act == "silu" else torch.sigmoid(-c * (g + CUBE * g ** 3))  # 1 - p
    return g * p, p + g * p * q * slope


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


class Made:
    def __init__(self, m, n, k, seed=0, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        kb, nb = -(-k // 128), -(-n // 128)
        self.m, self.n, self.k = m, n, k
        self.a, self.sa = random_codes((m, k), g), torch.exp(0.5 * torch.randn(m, kb, generator=g))
        self.w = [(random_codes((n, k), g), torch.exp(0.5 * torch.randn(nb, kb, generator=g)) * gain / (2e4 * k ** 0.5)) for _ in range(2)]
        v = plain64.value(self.a)
        (self.g, self.g_mag), (self.u, self.u_mag) = (plain64.product(v, self.sa, plain64.value(w), s, 128) for w, s in self.w)

    def hidden(self, act):
        """H and its tolerance before rounding."""
        a, _ = act64(self.g, act)
        h = a * self.u
        return h, 1.2e-5 * self.g_mag * self.u.abs() + 1e-5 * self.u_mag * self.g.abs() + 1.2e-10 * self.g_mag * self.u_mag + 2.0 ** -18 * h.abs()

    def run(self, h, nk, act, out, keep, stream=None):
        w = [t.to(DEV) for pair in self.w for t in pair] if nk else [t.t().contiguous().to(DEV) for pair in self.w for t in pair]
        a, sa = self.a.to(DEV), self.sa.to(DEV)
        sH = None
        if out == "e4m3":
            H = torch.full((self.m, self.n), 0x7F, dtype=torch.uint8, device=DEV)
            sH = torch.full((self.m, -(-self.n // 128)), math.nan, device=DEV)
        else:
            H = torch.full((self.m, self.n), math.nan, dtype=torch.float32 if out == "f32" else torch.bfloat16, device=DEV)
        kept = [torch.full((self.m, self.n), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2)] if keep else [None, None]
        mx.mxgemm_run_gated_block128(h, self.m, self.n, self.k, a, sa, w[0], w[1], w[2], w[3], H, H_scale=sH, act=ACTS[act],
                                     out_dtype={"f32": mx.OUT_F32, "bf16": mx.OUT_BF16, "e4m3": mx.OUT_E4M3}[out], gate=kept[0],
                                     up=kept[1], stream=stream)
        torch.cuda.synchronize()
        assert mx.mxgemm_get_device_status(h) == (0, 0)
        return H.cpu(), None if sH is None else sH.cpu(), [None if t is None else t.cpu() for t in kept]


def near(x, ref, tol, what):
    assert torch.isfinite(x.double()).all(), what
    err = (x.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: worst {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"


def check_codes(codes, scales, ref, tol, what):
    """Codes and scales by rows of 128, of values `ref` known to `tol`."""
    r, c = ref.shape
    pad = lambda t: torch.nn.functional.pad(t, (0, -c % 128)).view(r, -1, 128)  # noqa: E731
    top, most = pad(ref.abs()).amax(2), pad(tol).amax(2)
    near(scales, top.clamp(min=2.0 ** -100) / 448, most / 448 + 2.0 ** -23 * top + 2.0 ** -120, what + " scales")
    s = scales.double().repeat_interleave(128, 1)[:, :c]
    value = plain64.value(codes) * s
    # (the value that was rounded is off by tol, and by 2^-22 in the reciprocal and the product)
    near(value, ref, 2.0 ** -4 * ref.abs() * 1.001 + 2.0 ** -10 * s + 1.07 * tol, what)


def check(made, act, out, keep, got):
    H, sH, kept = got
    ref, tol = made.hidden(act)
    if out == "e4m3":
        check_codes(H, sH, ref, tol, "H")
    else:
        near(H, ref, tol * 1.01 + (2.0 ** -8 * ref.abs() if out == "bf16" else 0) + 1e-38, "H")
    if keep:
        for x, y, mag, name in ((kept[0], made.g, made.g_mag, "gate"), (kept[1], made.u, made.u_mag, "up")):
            near(x, y, 1.01e-5 * mag + 2.0 ** -8 * y.abs(), name)


SHAPES = [  # m, n, k: one row, ragged columns, K of one partial block, several CTAs for a column block, every width of M
    (1, 16, 16), (1, 272, 400), (5, 128, 2048), (16, 1000, 1040), (17, 512, 96), (33, 144, 4096), (64, 400, 528),
    (65, 16, 144), (100, 272, 256), (130, 128, 4112), (256, 1024, 128), (300, 528, 1168), (513, 784, 384), (700, 304, 2064),
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward(handles, m, n, k, nk, act):
    n = n if nk else -(-n // 16) * 16
    made = Made(m, n, k, m + n + k)
    for out in ("f32", "bf16", "e4m3"):
        if out == "e4m3" and n % 16:
            continue
        for keep in (False, True):
            check(made, act, out, keep, made.run(handles[nk], nk, act, out, keep))


@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (3, 130, 256), (40, 7, 272), (64, 999, 128), (66, 1, 32), (300, 257, 272), (260, 1001, 384)])
def test_odd_columns(handles, m, n, k):
    made = Made(m, n, k, 3)
    for out in ("f32", "bf16"):
        check(made, "silu", out, True, made.run(handles[True], True, "silu", out, True))


@pytest.mark.parametrize("m,n,k", [(16, 4000, 4096), (64, 2048, 8192), (600, 1536, 8192), (2600, 1200, 1024)])
def test_split_column_blocks_and_tiles(handles, m, n, k):
    """Column blocks that several CTAs share, tiles whose K is cut: equal bits again."""
    made = Made(m, n, k, 5)
    for out in ("e4m3", "bf16"):
        one = made.run(handles[True], True, "silu", out, True)
        check(made, "silu", out, True, one)
        two = made.run(handles[True], True, "silu", out, True)
        assert torch.equal(one[0], two[0]) and all(torch.equal(x, y) for x, y in zip(one[2], two[2]))
        assert out != "e4m3" or torch.equal(one[1], two[1])


@pytest.mark.parametrize("m", [8, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_gates(handles, m, act):
    """Gates of some hundreds: the activation is 0 or its argument there."""
    made = Made(m, 256, 256, 7, gain=60.0)
    assert float(made.g.abs().max()) > 150
    check(made, act, "f32", True, made.run(handles[True], True, act, "f32", True))


@pytest.mark.parametrize("m", [4, 200])
def test_rows_of_zeros(handles, m):
    made = Made(m, 160, 256, 8)
    made.a[1] = 0
    made.g[1] = made.u[1] = made.g_mag[1] = made.u_mag[1] = 0
    H, sH, _ = got = made.run(handles[True], True, "silu", "e4m3", False)
    check(made, "silu", "e4m3", False, got)
    assert (H[1] & 0x7F == 0).all() and (sH[1] == 2.0 ** -100 / 448).all()


@pytest.mark.parametrize("m", [12, 140])
def test_e5m2_operands(handles, m):
    h = handles[True]
    made = Made(m, 272, 400, 9)
    g = torch.Generator().manual_seed(2)
    finite = lambda shape: torch.randint(0, 0x60, shape, generator=g).to(torch.uint8) | (torch.randint(0, 2, shape, generator=g) << 7).to(torch.uint8)  # noqa: E731
    made.a = finite((m, 400))
    (made.g, made.g_mag), (made.u, made.u_mag) = (plain64.product(plain64.value_e5m2(made.a), made.sa, plain64.value(w), s, 128) for w, s in made.w)
    mx.mxgemm_set_option(h, mx.OPT_A_FORMAT, mx.FMT_E5M2)
    try:
        check(made, "silu", "f32", False, made.run(h, True, "silu", "f32", False))
    finally:
        mx.mxgemm_set_option(h, mx.OPT_A_FORMAT, mx.FMT_E4M3)


@pytest.mark.parametrize("m,out", [(16, "e4m3"), (16, "bf16"), (300, "e4m3"), (300, "bf16"), (2600, "e4m3")])
@pytest.mark.parametrize("stall", [1, 2, 3, 4])
def test_a_call_that_gives_up_leaves_nothing(m, out, stall):
    """A stalled producer: the status says so, and the next call is right again."""
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
    made = Made(m, 656, 2048, 11)
    good = made.run(h, True, "silu", out, False)
    mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000)
    mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, stall)
    H, sH = torch.zeros(m, 656, dtype=torch.uint8 if out == "e4m3" else torch.bfloat16, device=DEV), torch.zeros(m, 6, device=DEV)
    a, sa, (g, sg), (u, su) = made.a.to(DEV), made.sa.to(DEV), *[(w.to(DEV), s.to(DEV)) for w, s in made.w]
    mx.mxgemm_run_gated_block128(h, m, 656, 2048, a, sa, g, sg, u, su, H, H_scale=sH if out == "e4m3" else None,
                                 out_dtype=mx.OUT_E4M3 if out == "e4m3" else mx.OUT_BF16)
    torch.cuda.synchronize()
    assert mx.mxgemm_get_device_status(h)[0] == mx.ERR_TIMEOUT
    mx.mxgemm_set_option(h, mx.OPT_TEST_STALL_PRODUCER, 0)
    mx.mxgemm_set_option(h, mx.OPT_WAIT_TIMEOUT_NS, 2_000_000_000)
    again = made.run(h, True, "silu", out, False)
    assert torch.equal(good[0], again[0])
    mx.mxgemm_destroy(h)


def test_of_the_single_products(handles):
    """g and u are what the single product gives, to its tolerance, and H as codes what
    the quantizer makes of H in FP32 (equal, or a step apart where the sums' order differs)."""
    h = handles[True]
    made = Made(200, 384, 1024, 21)
    H, sH, kept = made.run(h, True, "gelu", "e4m3", True)
    for i in range(2):
        C = torch.empty(200, 384, dtype=torch.bfloat16, device=DEV)
        w, s = (t.to(DEV) for t in made.w[i])
        mx.mxgemm_run_block128(h, 200, 384, 1024, made.a.to(DEV), made.sa.to(DEV), w, s, C, out_dtype=mx.OUT_BF16)
        near(C.cpu(), kept[i].double(), 2.0 ** -7 * kept[i].double().abs() + 2e-5 * (made.g_mag, made.u_mag)[i], "product")
    F, _, _ = made.run(h, True, "gelu", "f32", False)
    codes, scales = torch.empty(200, 384, dtype=torch.uint8, device=DEV), torch.empty(200, 3, device=DEV)
    mx.mxgemm_quantize_block128(F.to(DEV), 200, 384, codes, scales)
    assert torch.equal(codes.cpu(), H) and torch.equal(scales.cpu(), sH)


# ---------------------------------------------------------------- the gradient
def grads64(g, u, dh, act):
    a, slope = act64(g.double(), act)
    dg, du, h = dh.double() * u.double() * slope, dh.double() * a, a * u.double()
    # p and a (1 - p) slope are of the order of 1 and cancel in part: 2^-18 of their sizes
    size = dh.double().abs() * u.double().abs()
    tol = 2.0 ** -18
    return {"dgate": (dg, tol * size * (1 + slope.abs())), "dup": (du, tol * du.abs()), "hidden": (h, tol * h.abs())}


def backward(g, u, dh, act, want, tall):
    r, c = g.shape
    out = {}
    for name in want:
        if name in ("dgate", "dup"):
            out[name] = torch.full((r, c), math.nan, dtype=torch.bfloat16, device=DEV)
        else:
            shape, blocks = ((r, c), (r, -(-c // 128))) if name.endswith("rows") else ((c, tall), (c, -(-r // 128)))
            out[name] = (torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV), torch.full(blocks, math.nan, device=DEV))
    mx.mxgemm_gated_backward(g.to(DEV), u.to(DEV), dh.to(DEV), r, c, act=ACTS[act], **out)
    torch.cuda.synchronize()
    return {k: (v[0].cpu(), v[1].cpu()) if isinstance(v, tuple) else v.cpu() for k, v in out.items()}


def check_backward(got, g, u, dh, act):
    r, c = g.shape
    ref = grads64(g, u, dh, act)
    for name, x in got.items():
        y, tol = ref[name.split("_")[0]]
        tol = tol + 1e-38
        if name in ("dgate", "dup"):
            near(x, y, 1.01 * tol + 2.0 ** -8 * y.abs() + 2.0 ** -134, name)
        elif name.endswith("rows"):
            check_codes(*x, y, tol, name)
        else:
            assert (x[0][:, r:] == 0).all()
            check_codes(x[0][:, :r].contiguous(), x[1], y.t().contiguous(), tol.t().contiguous(), name)


ALL = ["dgate", "dup", "dgate_rows", "dup_rows", "dgate_cols", "dup_cols", "hidden_cols"]


def inputs(r, c, x, seed=0):
    g = torch.Generator().manual_seed(seed)
    dh = torch.randn(r, c, generator=g) * torch.exp(torch.randn(r, 1, generator=g)) * 1e-3
    return [(2 * torch.randn(r, c, generator=g)).bfloat16() for _ in range(2)] + [dh.to(torch.bfloat16 if x == "bf16" else torch.float32)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("r,c", [(1, 16), (1, 128), (3, 144), (16, 32), (17, 272), (127, 128), (128, 112), (129, 256), (300, 1040), (1000, 400)])
def test_backward(r, c, x, act):
    g, u, dh = inputs(r, c, x, r + c)
    tall = -(-r // 16) * 16
    every = backward(g, u, dh, act, ALL, tall)
    check_backward(every, g, u, dh, act)
    for name in ALL:  # each by itself: the same
        one = backward(g, u, dh, act, [name], tall)[name]
        if isinstance(one, tuple):
            assert torch.equal(one[0], every[name][0]) and torch.equal(one[1], every[name][1])
        else:
            assert torch.equal(one, every[name])


@pytest.mark.parametrize("r,c", [(1, 1), (3, 5), (7, 129), (1741, 77), (64, 1000)])
def test_backward_of_any_size(r, c):
    for x in ("bf16", "f32"):
        g, u, dh = inputs(r, c, x)
        check_backward(backward(g, u, dh, "silu", ["dgate", "dup"], 0), g, u, dh, "silu")


def test_backward_far_gates_and_zeros():
    g, u, dh = inputs(64, 128, "f32")
    g[:8] *= 200
    g[8:12], u[12:16], dh[16:20] = 0, 0, 0
    g[20], g[21] = 3e38, -3e38
    for act in ACTS:
        got = backward(g, u, dh, act, ["dgate", "dup"], 64)
        # (a gate of 3e38 is past what its activation's values can be multiplied with)
        assert torch.isfinite(got["dgate"].float()).all() and not torch.isnan(got["dup"]).any()
        keep = torch.ones(64, dtype=torch.bool)
        keep[20:22] = False
        check_backward({k: v[keep] for k, v in got.items()}, g[keep], u[keep], dh[keep], act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_against_differences(act):
    """dgate and dup from differences of the kernel's definition in 64 bits."""
    g, u, dh = inputs(40, 64, "f32", 3)
    got = backward(g, u, dh, act, ["dgate", "dup"], 0)
    e = 1e-5
    f = lambda a, b: dh.double() * act64(a, act)[0] * b  # noqa: E731
    gd, ud = g.double(), u.double()
    num = {"dgate": (f(gd + e, ud) - f(gd - e, ud)) / (2 * e), "dup": (f(gd, ud + e) - f(gd, ud - e)) / (2 * e)}
    for name, y in num.items():  # (central differences: e^2 times the third derivative, and 2^-53 / e)
        near(got[name], y, 2.0 ** -8 * y.abs() + 1e-7 * dh.double().abs() * (1 + ud.abs() + gd.abs()), name)


def test_forward_and_backward_in_graphs(handles):
    """Captured and replayed, the capture's own launches and another stream."""
    h = handles[True]
    made = Made(40, 272, 512, 31)
    w = [t.to(DEV) for pair in made.w for t in pair]
    a, sa = made.a.to(DEV), made.sa.to(DEV)
    H, sH = torch.zeros(40, 272, dtype=torch.uint8, device=DEV), torch.zeros(40, 3, device=DEV)
    kept = [torch.zeros(40, 272, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    dh = torch.randn(40, 272, device=DEV)
    d = [torch.zeros(40, 272, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def step(stream):
        mx.mxgemm_run_gated_block128(h, 40, 272, 512, a, sa, *w, H, H_scale=sH, out_dtype=mx.OUT_E4M3, gate=kept[0], up=kept[1], stream=stream)
        mx.mxgemm_gated_backward(kept[0], kept[1], dh, 40, 272, dgate=d[0], dup=d[1], stream=stream)

    side = torch.cuda.Stream()
    step(side)
    side.synchronize()
    want = [t.clone() for t in (H, sH, *kept, *d)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(torch.cuda.current_stream())
    for t in (H, sH, *kept, *d):
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, (H, sH, *kept, *d)))


def test_launches_are_counted(handles):
    h = handles[True]
    n = mx.mxgemm_get_launch_count(h)
    made = Made(8, 64, 64)
    made.run(h, True, "silu", "f32", False)
    assert mx.mxgemm_get_launch_count(h) == n + 1
