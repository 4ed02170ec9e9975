"""The gradients of a linear layer through the quantizer and the product, as whole
matrices and along directions.

E4M3 rounds a value by 2^-4 of itself at most, by 0.027 of it in root mean square
(uniform over a binade's steps); both operands of a product are rounded, independently:
0.038 of the product's norm, and 0.08 is allowed.  Along the gradient itself, D = G,
the derivative's error is then at most 0.08 |G|^2, and along a direction of independent
normal values it is normal with 0.038 |G|: five times that is allowed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"
ALLOWED = 0.08


def near(got, want):
    """As a whole, and each row and column of some size by what independent errors leave."""
    off = (got - want).norm(dim=1) <= 2 * ALLOWED * want.norm(dim=1) + ALLOWED * want.norm() / want.shape[0] ** 0.5
    return bool((got - want).norm() <= ALLOWED * want.norm()) and bool(off.all())


def along(got, want, d, slope):
    """The derivative along d, from differences, against the gradient's."""
    mine = float((got * d).sum())
    return abs(mine - slope) <= 5 * 0.038 * float(want.norm()) * float(d.std()) if d is not want else abs(mine - slope) <= ALLOWED * slope


@pytest.fixture(scope="module")
def handles():
    hs = {}
    for nk in (True, False):
        hs[nk] = mx.mxgemm_create(0)
        mx.mxgemm_set_option(hs[nk], mx.OPT_B_MAJOR, mx.B_N_BY_K if nk else mx.B_K_BY_N)
    yield hs
    for h in hs.values():
        mx.mxgemm_destroy(h)


def quantized(t, block):
    r, c = t.shape
    shape = {"rows": (r, -(-c // 128)), "cols": (c, -(-r // 128)), "tiles": (-(-r // 128), -(-c // 128))}[block]
    codes = torch.empty((c, -(-r // 16) * 16) if block == "cols" else (r, c), dtype=torch.uint8, device=DEV)
    scales = torch.empty(shape, device=DEV)
    mx.mxgemm_quantize_block128(t.to(DEV), r, c, codes, scales, block={"rows": mx.BLOCK_ROWS, "cols": mx.BLOCK_COLS, "tiles": mx.BLOCK_TILES}[block])
    return codes, scales


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,I,O", [(300, 272, 400), (40, 512, 256), (513, 144, 1040)])
def test_gradients(handles, T, I, O, dtype):
    g = torch.Generator().manual_seed(T)
    x, w, dy = (t.to(dtype) for t in (torch.randn(T, I, generator=g), torch.randn(O, I, generator=g) * 0.05, torch.randn(T, O, generator=g) * 0.01))
    (cw, sw), (cy, sy) = quantized(w, "tiles"), quantized(dy, "rows")
    dx = torch.empty(T, I, device=DEV)
    mx.mxgemm_run_block128(handles[False], T, I, O, cy, sy, cw, sw, dx)
    (ca, sa), (cb, sb) = quantized(dy, "cols"), quantized(x, "cols")
    dw = torch.empty(O, I, device=DEV)
    mx.mxgemm_run_block128(handles[True], O, I, ca.shape[1], ca, sa, cb, sb, dw, b_block=1)
    dx, dw = dx.cpu().double(), dw.cpu().double()
    x, w, dy = x.double(), w.double(), dy.double()
    want_dx, want_dw = dy @ w, dy.t() @ x
    loss = lambda x, w: float((dy * (x @ w.t())).sum())
    for got, want, moved in ((dx, want_dx, lambda d: (x + d, w)), (dw, want_dw, lambda d: (x, w + d))):
        assert near(got, want)
        directions = [want] + [torch.randn(want.shape, generator=g, dtype=torch.float64) for _ in range(3)]
        for d in directions:
            h = 1e-3 / float(d.norm())
            slope = (loss(*moved(h * d)) - loss(*moved(-h * d))) / (2 * h)  # the loss is linear in each: no error of second order
            assert along(got, want, d, slope)
        # what these checks are for: no gradient, one of the other sign, a row's, a factor's absence
        rows = want.clone()
        rows[want.shape[0] // 2] = 0
        for wrong in (torch.zeros_like(want), -want, 0.9 * want, rows):
            assert not near(wrong, want)
        slope = float(want.norm()) ** 2
        assert not along(torch.zeros_like(want), want, want, slope) and not along(-want, want, want, slope)
