"""What the calls of a transformer layer's parts refuse, without a GPU: the library's
checks that come before any device is asked, the binding's, and the frequencies."""
import math

import pytest
import torch

mx = pytest.importorskip("block_scaled_gemm_gb300")


def test_gated_without_a_handle():
    st = mx.mxgemm_run_gated_block128(None, 1, 16, 16, None, None, None, None, None, None, None, check=False)
    assert st == mx.ERR_INVALID_VALUE


def grads(r=4, c=32, x=torch.bfloat16, check=False, **kw):
    a = torch.zeros(r, c, dtype=torch.bfloat16)
    return mx.mxgemm_gated_backward(a, a, torch.zeros(r, c, dtype=x), r, c, check=check, **kw)


def test_gated_backward_refuses():
    """(Whole arguments are refused too, for their host pointers or for want of a GPU.)"""
    bf = torch.zeros(4, 32, dtype=torch.bfloat16)
    assert grads() == mx.ERR_INVALID_VALUE  # nothing is asked for
    assert grads(dgate=bf) in (mx.ERR_INVALID_VALUE, mx.ERR_CUDA)
    assert grads(dgate_rows=(bf, None)) == mx.ERR_INVALID_VALUE
    assert grads(dgate_rows=(None, bf)) == mx.ERR_INVALID_VALUE
    assert grads(c=24, dgate_rows=(bf, bf)) == mx.ERR_INVALID_VALUE
    assert grads(dgate=bf, act=2) == mx.ERR_INVALID_VALUE
    assert grads(dgate=bf, x_dtype=2) == mx.ERR_INVALID_VALUE
    assert grads(dgate=bf.data_ptr() + 2) == mx.ERR_MISALIGNED
    assert grads(dgate_cols=(bf.data_ptr() + 8, bf)) == mx.ERR_MISALIGNED
    assert grads(r=0, c=32, dgate=bf) == mx.OK and grads(r=4, c=0, dgate=bf) == mx.OK
    with pytest.raises(mx.MxgemmError, match="mxgemm_gated_backward"):
        grads(check=True)
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match="float32 or bfloat16"):
            grads(x=dtype, dgate=bf)


def test_gated_binding_refuses():
    f, b, c = torch.zeros(16, 16), torch.zeros(16, 16, dtype=torch.bfloat16), torch.zeros(16, 16, dtype=torch.uint8)
    call = lambda H, **kw: mx.mxgemm_run_gated_block128(None, 16, 16, 16, c, f, c, f, c, f, H, check=False, **kw)  # noqa: E731
    for H, out in ((b, mx.OUT_F32), (f, mx.OUT_BF16), (b, mx.OUT_E4M3), (c, mx.OUT_BF16), (b, 7)):
        with pytest.raises(ValueError):
            call(H, out_dtype=out)
    for kw in (dict(gate=f, up=b), dict(gate=b, up=c), dict(gate=b.half(), up=b)):
        with pytest.raises(ValueError):
            call(b, **kw)
    assert call(b, gate=b, up=b) == call(c, out_dtype=mx.OUT_E4M3, H_scale=f) == mx.ERR_INVALID_VALUE  # no handle
    for wrong in (dict(gate=f, up=b, dgate=b), dict(gate=b, up=b.half(), dgate=b), dict(gate=b, up=b, dgate=f), dict(gate=b, up=b, dup=c)):
        with pytest.raises(ValueError):
            mx.mxgemm_gated_backward(wrong.pop("gate"), wrong.pop("up"), b, 16, 16, check=False, **wrong)


def rope(q=None, k=None, **kw):
    q = torch.zeros(3, 2, 64) if q is None else q
    return mx.mxgemm_norm_rope(q, k, torch.zeros(q.shape, dtype=q.dtype), None if k is None else torch.zeros_like(k), check=False, **kw)


POS = torch.zeros(3, dtype=torch.int32)
F = torch.ones(32, dtype=torch.float64)


def test_rope_refuses():
    ok = dict(positions=POS, freqs=F)
    assert rope(**ok) == mx.ERR_INVALID_VALUE  # host memory
    assert rope(torch.zeros(0, 2, 64), positions=POS[:0], freqs=F) == mx.OK
    for bad in (torch.zeros(3, 2, 32), torch.zeros(3, 2, 96), torch.zeros(3, 2, 256)):
        assert rope(bad, **ok) == mx.ERR_INVALID_VALUE
    for n in (4, 12, 33, 40):  # rot no multiple of 16, or more than a head
        assert rope(positions=POS, freqs=torch.ones(n, dtype=torch.float64)) == mx.ERR_INVALID_VALUE
    for eps in (-1.0, math.nan, math.inf):
        assert rope(eps=eps, **ok) == mx.ERR_INVALID_VALUE
    for factor in (math.nan, math.inf):
        assert rope(factor=factor, **ok) == mx.ERR_INVALID_VALUE
    wide = torch.zeros(3, 2 * 64 + 4)[:, :128].view(3, 2, 64)
    assert rope(wide, **ok) == mx.ERR_MISALIGNED


def test_rope_binding_refuses():
    for kw in (dict(positions=POS.long(), freqs=F), dict(positions=POS[:2], freqs=F), dict(freqs=F), dict(positions=POS, freqs=F.float()),
               dict(q_weight=torch.ones(32)), dict(q_weight=torch.ones(64).double()), dict(q_weight=torch.ones(128)[::2])):
        with pytest.raises(ValueError):
            rope(**kw)
    with pytest.raises(ValueError):
        rope(torch.zeros(3, 2, 64).half())
    with pytest.raises(ValueError):
        rope(torch.zeros(3, 64, 2).transpose(1, 2))
    with pytest.raises(ValueError):
        rope(k=torch.zeros(3, 2, 64).bfloat16())
    with pytest.raises(ValueError):
        rope(k=torch.zeros(4, 2, 64))
    with pytest.raises(ValueError):
        rope(k=torch.zeros(3, 2, 64), q_weight=torch.ones(64), k_weight=torch.ones(64).bfloat16())
    q = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):  # a result of another type
        mx.mxgemm_norm_rope(q, None, q.bfloat16(), None)
    with pytest.raises(ValueError):  # a norm's gradient without the values
        mx.mxgemm_norm_rope_backward(None, q, None, q.clone(), None, q_weight=torch.ones(64))
    with pytest.raises(ValueError):  # a weight's gradient without a weight
        mx.mxgemm_norm_rope_backward(None, q, None, q.clone(), None, q=q, dq_weight=torch.ones(64))


def test_keys_without_a_result_are_refused():
    q, k, w = torch.zeros(3, 2, 64), torch.zeros(3, 1, 64), torch.ones(64)
    for args, kw in (((q, k, q, None), {}), ((q, None, None, None), {})):
        with pytest.raises(ValueError):
            mx.mxgemm_norm_rope(*args, **kw)
    for args, kw in (((q, k, q, None), {}), ((q, None, q, None), dict(k=k)), ((q, None, q, None), dict(dk_weight=w)), ((q, None, None, None), {})):
        with pytest.raises(ValueError):
            mx.mxgemm_norm_rope_backward(None, *args, **kw)
    # a weight alone asks for nothing
    assert mx.mxgemm_norm_rope(q[:0], None, q[:0], None, k_weight=w) == mx.OK


def test_handles_are_needed():
    q = torch.zeros(3, 2, 64)
    assert mx.mxgemm_norm_rope_backward(None, q, None, q.clone(), None, check=False) == mx.ERR_INVALID_VALUE
    codes, scales = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(3, 2)
    cache = mx.Cache(codes, codes.clone(), scales, scales.clone())
    b = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    assert mx.mxgemm_cache_attention_shared(None, cache, table, lens, 16, b, b.clone(), check=False) == mx.ERR_INVALID_VALUE
    with pytest.raises(ValueError):
        mx.mxgemm_cache_attention_shared(None, cache, table.long(), lens, 16, b, b.clone())
    with pytest.raises(ValueError):
        mx.mxgemm_cache_attention_shared(None, cache, table, lens, 16, b.float(), b.clone())


# ---------------------------------------------------------------- frequencies
def test_plain_frequencies():
    f = mx.mxgemm_rope_frequencies(64, 10000.0)
    j = torch.arange(32, dtype=torch.float64)
    assert f.dtype is torch.float64 and torch.allclose(f, 10000.0 ** (-j / 32), rtol=1e-14, atol=0)
    assert mx.mxgemm_rope_frequencies(0).numel() == 0


def test_stretched_frequencies():
    f = mx.mxgemm_rope_frequencies(64, 10000.0)
    assert torch.allclose(mx.mxgemm_rope_frequencies(64, 10000.0, mx.ROPE_LINEAR, 8.0), f / 8, rtol=1e-14, atol=0)
    g = mx.mxgemm_rope_frequencies(64, 10000.0, mx.ROPE_BASE, 8.0)
    assert math.isclose(float(g[0]), 1.0) and math.isclose(float(g[-1]), float(f[-1]) / 8, rel_tol=1e-12)
    p = mx.mxgemm_rope_frequencies(64, 10000.0, mx.ROPE_BY_PARTS, 8.0, trained=4096, slow=1.0, fast=32.0)
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    assert torch.allclose(p, f / 8 * (1 - keep) + f * keep, rtol=1e-13, atol=0)
    assert (p[turns >= 32] == f[turns >= 32]).all() and torch.allclose(p[turns <= 1], f[turns <= 1] / 8, rtol=1e-14, atol=0)
    assert (keep > 0).any() and (keep < 1).any() and ((keep > 0) & (keep < 1)).any()


@pytest.mark.parametrize("args", [(63,), (-2,), (64, 0.0), (64, -1.0), (64, math.inf), (64, math.nan), (64, 1e4, 4), (64, 1e4, -1),
                                  (64, 1e4, mx.ROPE_LINEAR, 0.5), (64, 1e4, mx.ROPE_LINEAR, math.nan), (2, 1e4, mx.ROPE_BASE, 2.0),
                                  (64, 1e4, mx.ROPE_BY_PARTS, 2.0), (64, 1e4, mx.ROPE_BY_PARTS, 2.0, 4096, 4.0, 4.0),
                                  (64, 1e4, mx.ROPE_BY_PARTS, 2.0, 4096, 0.0, 4.0)])
def test_frequencies_refuse(args):
    with pytest.raises(mx.MxgemmError):
        mx.mxgemm_rope_frequencies(*args)
