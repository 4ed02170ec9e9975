"""H of a gated pair of products in FP32 is to FP32's precision, for gates near and far
from 0.  Operands of one nonzero code make g and u exact, so that what is off is the
activation alone, in units of 2^-24 of it: 2^t 4 units, the first-order term of the rest
of the argument 1, its FP32 ln 2 (2^-25 of itself or less, times 88) 4, the sum 1, the
reciprocal 2, two products 1 each: 14 units, 2^-20.2.  GELU's argument z is off by four
roundings, 2^-22 of itself, and so is e^z by 2^-22 |z|."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"
ONE, MINUS = 0x38, 0xB8  # E4M3 codes


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m", [1, 13, 40, 64, 65, 300])
def test_exact_gates(m, act):
    n = 272
    g = torch.Generator().manual_seed(m)
    A = torch.zeros(m, 16, dtype=torch.uint8)
    A[:, 3] = ONE
    most = 88.0 if act == "silu" else 9.5  # e^-2z stays in FP32's range
    # magnitudes of the rows' gates from 2^-20 to `most`; the scale of A is the gate
    sA = (torch.rand(m, 1, generator=g) * (math.log2(most) + 20) - 20).exp2().clamp(max=most * 0.985)
    G = torch.zeros(n, 16, dtype=torch.uint8)
    G[:, 3] = torch.where(torch.arange(n) % 2 == 0, ONE, MINUS).to(torch.uint8)
    U = torch.zeros(n, 16, dtype=torch.uint8)
    U[:, 3] = ONE
    sG, sU = torch.ones(3, 1), torch.tensor([[1.0], [0.5], [2.0]])
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
    H = torch.empty(m, n, device=DEV)
    dev = [t.to(DEV) for t in (A, sA, G, sG, U, sU)]
    mx.mxgemm_run_gated_block128(h, m, n, 16, *dev, H, act=mx.ACT_SILU if act == "silu" else mx.ACT_GELU_TANH, out_dtype=mx.OUT_F32)
    torch.cuda.synchronize()
    x = sA.double() * torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)
    u = sA.double() * sU.double().repeat_interleave(128)[:n]
    z = x if act == "silu" else 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    want = x * torch.sigmoid(z) * u
    tol = 2.0 ** -20.2 + (0 if act == "silu" else 2.0 ** -22 * z.abs())
    off = ((H.cpu().double() - want).abs() / (tol * want.abs())).max().item()
    assert off <= 1, f"{off} of the tolerance"
    mx.mxgemm_destroy(h)
