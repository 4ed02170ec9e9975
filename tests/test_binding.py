"""Checks of the Python binding that need no GPU: what it refuses before a call."""
import pytest
import torch

mx = pytest.importorskip("block_scaled_gemm_gb300")


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, torch.uint8, torch.float8_e4m3fn])
@pytest.mark.parametrize("quantize", ["mxgemm_quantize", "mxgemm_quantize_block128"])
def test_quantizers_refuse_other_types(quantize, dtype):
    """They read 4 bytes a value unless X is bfloat16: an FP16 X has half of that."""
    x = torch.zeros(64, 64).to(dtype)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        getattr(mx, quantize)(x, 64, 64, torch.zeros(4096, dtype=torch.uint8), torch.zeros(64), check=False)


@pytest.mark.parametrize("quantize", ["mxgemm_quantize", "mxgemm_quantize_block128"])
def test_quantizers_take_their_types_and_addresses(quantize):
    """Refused by the library for other reasons (no device pointers)."""
    for x in (torch.zeros(64, 64), torch.zeros(64, 64).bfloat16(), None):
        assert getattr(mx, quantize)(x, 64, 64, None, None, check=False) == mx.ERR_INVALID_VALUE


def test_cache_refuses_other_scales_and_codes():
    codes, scales = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(3, 2)
    mx.Cache(codes, codes.clone(), scales, scales.clone())
    f8 = codes.view(torch.float8_e4m3fn)
    mx.Cache(f8, f8.clone(), scales, scales.clone())
    for wrong in (scales.int(), scales.view(torch.int32), scales.double(), scales.half()):
        for pair in ((wrong, scales), (scales, wrong), (wrong, wrong)):
            with pytest.raises(ValueError):
                mx.Cache(codes, codes, *pair)
    e5, z = codes.view(torch.float8_e5m2), codes.view(torch.float8_e4m3fnuz)
    for pair in ((e5, codes), (codes, e5), (z, z), (codes.half(), codes.half())):
        with pytest.raises(ValueError):
            mx.Cache(*pair, scales, scales)
