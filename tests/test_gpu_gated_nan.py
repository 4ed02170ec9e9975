"""NaN in H as codes stays where it is: the scale of its block and the block's other codes
are those of the values that are none, for few rows and for many, as the quantizer has it."""
import pytest
import torch

from test_gpu_gated import DEV, Made, mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nk", [True, False])
@pytest.mark.parametrize("m,n,k", [(1, 256, 128), (16, 400, 4096), (30, 144, 256), (64, 272, 400), (65, 256, 128), (300, 400, 272)])
@pytest.mark.parametrize("columns", [[5], [8, 9, 10, 11], [128, 129, 130, 131, 140]])
def test_nan_columns(m, n, k, nk, columns):
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K if nk else mx.B_K_BY_N)
    made = Made(m, n, k, m + n)
    made.w[0][0][columns] = 0  # products of 0
    want, scales, _ = made.run(h, nk, "silu", "e4m3", False)
    made.w[0][0][columns] = 0x7F
    H, sH, _ = made.run(h, nk, "silu", "e4m3", False)
    assert torch.equal(sH, scales)
    rest = torch.tensor([c not in columns for c in range(n)])
    assert torch.equal(H[:, rest], want[:, rest]) and ((H[:, ~rest] & 0x7F) == 0x7F).all()
    F, _, _ = made.run(h, nk, "silu", "f32", False)
    codes, s = torch.empty(m, n, dtype=torch.uint8, device=DEV), torch.empty_like(sH, device=DEV)
    mx.mxgemm_quantize_block128(F.to(DEV), m, n, codes, s)
    assert torch.equal(codes.cpu() & 0x7F, H & 0x7F) and torch.equal(s.cpu(), sH)
    mx.mxgemm_destroy(h)
