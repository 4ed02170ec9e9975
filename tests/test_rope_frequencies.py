"""Stretched frequencies whose base would not be finite are refused (they came out as 0)."""
import pytest

mx = pytest.importorskip("block_scaled_gemm_gb300")


def test_a_base_past_the_range():
    for rot, base, scale in ((4, 1e200, 1e60), (64, 1e300, 1e9), (4, 2.0, 1e200)):
        with pytest.raises(mx.MxgemmError):
            mx.mxgemm_rope_frequencies(rot, base, mx.ROPE_BASE, scale=scale)
    f = mx.mxgemm_rope_frequencies(4, 1e100, mx.ROPE_BASE, scale=1e50)
    assert f[0] == 1 and abs(f[1] / 1e-100 - 1) < 1e-9
