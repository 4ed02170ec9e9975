"""Norms of queries and keys with the rotation by positions, and the gradient, on the
GPU, against plain 64-bit implementations.

Tolerance of a result: FP32 throughout.  The norm's factor is off by the sum of
squares (D / 16 + 3 roundings of terms of one sign), a square root and a division,
2^-20 of itself; a value of the norm by 2^-19 with its products.  An angle is off by
2^-25 of half a turn (9.4e-8 rad) and the frequency's 2^-52 of the product (at most
2^31 radians: 3e-7 rad), sine and cosine by 2^-22 more: 1e-6 of a pair's size covers
both, and 1e-5 all.  A gradient's mean takes D products more, of sizes that may
cancel: 1e-5 of the sum of sizes.  BF16 adds 2^-8 of the value.  dweight: a sum of
tokens x heads terms in up to 64 + 25 + 25 steps a thread and a tree: 2^-24 * 128 of
the sum of sizes, and the terms' own 1e-5."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def h():
    h = mx.mxgemm_create(0)
    yield h
    mx.mxgemm_destroy(h)


def pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn64(x, positions, freqs, interleaved, factor, back=False):
    """(turned, sizes) in 64 bits; the angles' turns from exact integers of the frequencies' doubles."""
    y, size = x.clone(), x.abs()
    rot = 2 * freqs.numel()
    if rot:
        one, two = pairs(rot, interleaved)
        # angle mod 2 pi: split the frequency so that both products are exact enough
        w = positions.double()[:, None] * freqs[None]
        c, s = factor * torch.cos(w)[:, None], factor * torch.sin(w)[:, None] * (-1 if back else 1)
        y[..., one], y[..., two] = x[..., one] * c - x[..., two] * s, x[..., two] * c + x[..., one] * s
        size[..., one] = size[..., two] = abs(factor) * (x[..., one].abs() + x[..., two].abs())
    return y, size


def forward64(x, w, eps, *turn):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(2, keepdim=True) + eps) * w.double()
    return turn64(x, *turn)


def backward64(x, dy, w, eps, positions, freqs, interleaved, factor):
    dn, size = turn64(dy.double(), positions, freqs, interleaved, factor, True)
    if w is None:
        return dn, size, None, None
    x, w = x.double(), w.double()
    r = 1 / torch.sqrt(x.square().mean(2, keepdim=True) + eps)
    hat = x * r
    g = dn * w
    dx = r * (g - hat * (g * hat).mean(2, keepdim=True))
    gs = size * w.abs()
    dx_size = r * (gs + hat.abs() * (gs * hat.abs()).mean(2, keepdim=True))
    return dx, dx_size, (dn * hat).sum((0, 1)), (size * hat.abs()).sum((0, 1))


def near(x, ref, tol, what):
    x = x.cpu().double()
    assert torch.isfinite(x).all(), what
    err = (x - ref).abs()
    assert (err <= tol).all(), f"{what}: worst {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"


class Case:
    def __init__(self, tokens, hq, hk, d, rot, interleaved, dtype, norm, far=5000, wtype=torch.float32, factor=1.0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.tokens, self.d, self.interleaved, self.factor, self.dtype = tokens, d, interleaved, factor, dtype
        rows = (torch.randn(tokens, (hq + 2 * hk) * d, generator=g) * torch.exp(torch.randn(tokens, 1, generator=g))).to(dtype)
        self.rows = rows
        self.x = [rows[:, :hq * d].view(tokens, hq, d), rows[:, hq * d:(hq + hk) * d].view(tokens, hk, d)]
        self.dy = [torch.randn(tokens, n, d, generator=g).to(dtype) for n in (hq, hk)]
        self.w = [(1 + 0.2 * torch.randn(d, generator=g)).to(wtype) if norm else None for _ in range(2)]
        self.pos = torch.randint(0, far, (tokens,), generator=g, dtype=torch.int32)
        self.freqs = mx.mxgemm_rope_frequencies(rot) if rot else torch.zeros(0, dtype=torch.float64)
        self.eps = 1e-6

    def turn(self):
        return self.pos, self.freqs, self.interleaved, self.factor

    def on_device(self):
        rows = self.rows.to(DEV)
        hq, hk = self.x[0].shape[1], self.x[1].shape[1]
        d, t = self.d, self.tokens
        x = [rows[:, :hq * d].view(t, hq, d), rows[:, hq * d:(hq + hk) * d].view(t, hk, d)]
        kw = {"positions": self.pos.to(DEV), "freqs": self.freqs.to(DEV) if self.freqs.numel() else None, "interleaved": self.interleaved,
              "factor": self.factor, "eps": self.eps}
        for n, w in zip("qk", self.w):
            kw[n + "_weight"] = None if w is None else w.to(DEV)
        return rows, x, kw

    def forward(self, stream=None):
        rows, x, kw = self.on_device()
        out = [torch.full(v.shape, math.nan, dtype=self.dtype, device=DEV) for v in x]
        none = x[1].shape[1] == 0
        mx.mxgemm_norm_rope(x[0], None if none else x[1], out[0], None if none else out[1], stream=stream, **kw)
        torch.cuda.synchronize()
        return out

    def backward(self, h):
        rows, x, kw = self.on_device()
        dx = [torch.full(v.shape, math.nan, dtype=self.dtype, device=DEV) for v in x]
        dw = [None if w is None else torch.full((self.d,), math.nan, device=DEV) for w in self.w]
        dy = [v.to(DEV) for v in self.dy]
        none = x[1].shape[1] == 0
        mx.mxgemm_norm_rope_backward(h, dy[0], None if none else dy[1], dx[0], None if none else dx[1], q=x[0],
                                     k=None if none else x[1], dq_weight=dw[0], dk_weight=None if none else dw[1], **kw)
        torch.cuda.synchronize()
        assert mx.mxgemm_get_device_status(h) == (0, 0)
        return dx, dw

    def check(self, out):
        for y, x, w, name in zip(out, self.x, self.w, ("q", "k")):
            ref, size = forward64(x, w, self.eps, *self.turn())
            near(y, ref, 1e-5 * size + (2.0 ** -8 * ref.abs() if self.dtype is torch.bfloat16 else 0) + 1e-38, name)

    def check_backward(self, dx, dw):
        for i, name in enumerate("qk"):
            if not self.x[i].shape[1]:
                continue
            ref, size, w, w_size = backward64(self.x[i], self.dy[i], self.w[i], self.eps, *self.turn())
            near(dx[i], ref, 1e-5 * size + (2.0 ** -8 * ref.abs() if self.dtype is torch.bfloat16 else 0) + 1e-38, "d" + name)
            if w is not None:
                near(dw[i], w, 2e-5 * w_size + 1e-38, "dweight " + name)


CASES = [  # tokens, query heads, key heads, d, rot, interleaved
    (1, 1, 1, 128, 128, False), (1, 8, 2, 64, 64, True), (3, 5, 1, 128, 64, False), (7, 33, 3, 64, 32, True), (8, 40, 0, 128, 16, False),
    (9, 64, 8, 128, 128, True), (65, 7, 7, 64, 48, False), (300, 12, 4, 128, 96, True), (2500, 4, 1, 64, 64, False), (2437, 2, 1, 128, 32, True),
    (13, 3, 2, 128, 0, False),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,hq,hk,d,rot,interleaved", CASES)
def test_forward_and_backward(h, tokens, hq, hk, d, rot, interleaved, dtype, norm):
    c = Case(tokens, hq, hk, d, rot, interleaved, dtype, norm, seed=tokens + hq)
    c.check(c.forward())
    c.check_backward(*c.backward(h))


@pytest.mark.parametrize("interleaved", [True, False])
def test_factor_and_bf16_weights(h, interleaved):
    c = Case(40, 6, 2, 128, 64, interleaved, torch.float32, True, wtype=torch.bfloat16, factor=-1.3)
    c.check(c.forward())
    c.check_backward(*c.backward(h))


def test_far_positions():
    """Angles of millions of turns, with frequencies that divide them exactly, so that the
    answer is known without a reduction: f = 2 pi a / 2^20 as a double is off by 2^-53 of
    itself, which the positions carry to 2^31 * 2^-53 turns."""
    tokens = 64
    c = Case(tokens, 4, 1, 64, 64, False, torch.float32, False)
    g = torch.Generator().manual_seed(5)
    a = torch.randint(1, 2 ** 20, (32,), generator=g)
    c.freqs = a.double() * (2 * math.pi / 2 ** 20)
    c.pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (tokens,), generator=g).to(torch.int32)
    c.pos[:4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, -1], dtype=torch.int32)
    out = c.forward()
    turns = (c.pos.long()[:, None] * a[None]) % 2 ** 20  # exact
    w = turns.double() * (2 * math.pi / 2 ** 20)
    one, two = pairs(64, False)
    for y, x in zip(out, c.x):
        x = x.double()
        z = torch.zeros_like(x)
        cos, sin = torch.cos(w)[:, None], torch.sin(w)[:, None]
        z[..., one], z[..., two] = x[..., one] * cos - x[..., two] * sin, x[..., two] * cos + x[..., one] * sin
        size = x[..., one].abs() + x[..., two].abs()
        near(y, z, 1e-5 * torch.cat((size, size), 2) + 1e-38, "far")


def test_in_place_and_on_another_stream(h):
    """Results in the projection's own buffer; its values and the places behind stay."""
    c = Case(50, 6, 2, 128, 128, False, torch.bfloat16, True)
    want = c.forward()
    rows, x, kw = c.on_device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mx.mxgemm_norm_rope(x[0], x[1], x[0], x[1], stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    assert torch.equal(rows[:, 8 * 128:].cpu(), c.rows[:, 8 * 128:])
    dx, dw = c.backward(h)
    rows, x, kw = c.on_device()
    dy, dw2 = [v.to(DEV) for v in c.dy], [torch.empty(128, device=DEV) for _ in range(2)]
    mx.mxgemm_norm_rope_backward(h, dy[0], dy[1], dy[0], dy[1], q=x[0], k=x[1], dq_weight=dw2[0], dk_weight=dw2[1], **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(dx + dw, dy + dw2))


def test_rows_of_zeros_and_of_one_large_value(h):
    c = Case(12, 2, 1, 128, 128, False, torch.float32, True)
    c.rows[0] = 0
    c.rows[1, :128] = 0
    c.rows[1, 5] = 1e15
    c.check(c.forward())
    c.check_backward(*c.backward(h))


def test_no_tokens(h):
    w = torch.ones(64, device=DEV)
    e = torch.empty(0, 3, 64, device=DEV)
    dw = torch.full((64,), 7.0, device=DEV)
    mx.mxgemm_norm_rope(e, None, e, None, q_weight=w)
    mx.mxgemm_norm_rope_backward(h, e, None, e, None, q=e, q_weight=w, dq_weight=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_weights_gradient_is_the_same_every_time(h):
    c = Case(3000, 8, 2, 128, 128, False, torch.bfloat16, True)
    first = c.backward(h)
    c.check_backward(*first)
    for _ in range(3):
        again = c.backward(h)
        assert all(torch.equal(x, y) for x, y in zip(first[1], again[1]))


def test_gradient_against_differences(h):
    """Along a direction, of the definition in 64 bits."""
    c = Case(5, 3, 2, 64, 48, True, torch.float32, True, far=100)
    dx, dw = c.backward(h)
    g = torch.Generator().manual_seed(1)
    for i in range(2):
        x, w, dy = c.x[i].double(), c.w[i].double(), c.dy[i].double()
        vx, vw = torch.randn(x.shape, generator=g, dtype=torch.float64) * x.abs(), torch.randn(64, generator=g, dtype=torch.float64)
        e = 1e-6
        f = lambda s: float((forward64(x + s * vx, w + s * vw, c.eps, *c.turn())[0] * dy).sum())  # noqa: E731
        num = (f(e) - f(-e)) / (2 * e)
        got = float((dx[i].cpu().double() * vx).sum() + (dw[i].cpu().double() * vw).sum())
        assert abs(num - got) <= 1e-4 * float((dx[i].cpu().double() * vx).abs().sum() + (dw[i].cpu().double() * vw).abs().sum())


def test_captured_and_replayed_beside_other_calls(h):
    """The gradient's workspace and counters in two graphs of one handle, replayed in turn."""
    a, b = Case(200, 4, 1, 64, 64, False, torch.float32, True, seed=1), Case(900, 8, 2, 128, 64, True, torch.float32, True, seed=2)
    want = [c.backward(h) for c in (a, b)]
    graphs, outs, keep = [], [], []
    for c in (a, b):
        rows, x, kw = c.on_device()
        dy, dx = [v.to(DEV) for v in c.dy], [torch.zeros(v.shape, device=DEV) for v in c.x]
        dw = [torch.zeros(c.d, device=DEV) for _ in range(2)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mx.mxgemm_norm_rope_backward(h, dy[0], dy[1], dx[0], dx[1], q=x[0], k=x[1], dq_weight=dw[0], dk_weight=dw[1],
                                         stream=torch.cuda.current_stream(), **kw)
        graphs.append(graph)
        outs.append(dx + dw)
        keep.append((rows, dy, kw))
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (dx, dw), out in zip(want, outs):
        assert all(torch.equal(x, y) for x, y in zip(dx + dw, out))
