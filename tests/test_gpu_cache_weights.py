"""Many small weights beside a large one: a first key that takes most of the sum and has
no value, as the first tokens of long sequences do, and thousands of keys that have.
Tolerance as in test_gpu_cache.py: 2^-10 of sum p|v| for the weights' rounding (they keep
11 bits down to 2^-21 of the largest), which here is the output itself, and for weights
down to 2^-26 of the largest, off by 2^-32 of it, 2^-6 of that sum."""
import math

import pytest
import torch

import plain64
import test_gpu_cache as tc

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")


@pytest.fixture(scope="module")
def h():
    h = mx.mxgemm_create(0)
    yield h
    mx.mxgemm_destroy(h)


@pytest.mark.parametrize("bits,allowed", [(15.3, 2.0 ** -10), (18.3, 2.0 ** -10), (20.3, 2.0 ** -10), (26.3, 2.0 ** -6)])
@pytest.mark.parametrize("length,new,group,d,page", [(20000, None, 8, 128, 64), (7001, None, 16, 64, 16), (5000, 70, 1, 64, 64), (3000, 300, 4, 128, 128)])
def test_small_weights_count(h, length, new, group, d, page, bits, allowed):
    """Weights 2^-bits of the first key's; 15 bits and more are FP16's subnormal range,
    25 its end, for weights whose largest is 1."""
    m = tc.Made([length], 1, d, page, seed=length)
    m.sK.fill_(1.0)
    m.sV.fill_(2.0 ** -3)
    filled = m.K != 0x7F
    m.K = torch.where(filled, 0, m.K)
    first = m.table[0][0]
    m.K[first, 0, 0, 0] = 0x58  # 16
    m.V = torch.where(filled, 0x38, m.V)  # 1
    m.V[first, 0, 0] = 0
    n = new or 1
    q = torch.zeros(n, group, d)
    q[..., 0] = 1
    q = q.bfloat16()
    scale = bits * math.log(2.0) / 16
    news = None if new is None else [new]
    O, L = tc.attend(h, m, q, news, scale=scale)
    o, lse, mag, size = plain64.attention(plain64.value(m.K), m.sK, plain64.value(m.V), m.sV, m.table, m.kv_len, [0, n], q, scale)
    assert float(size.max()) < 64
    err = (O.double() - o).abs()
    tol = 2.0 ** -8 * o.abs() + allowed * mag
    assert (err <= tol).all(), f"worst {float((err / tol.clamp(min=1e-300)).max())} of the tolerance"
    assert ((L.double() - lse).abs() <= 2.0 ** -19 * (1 + size)).all()


@pytest.mark.parametrize("lens,news,kv,group,d,page", [([7] * 40, None, 8, 4, 64, 16), ([20] * 30, [8] * 30, 8, 8, 64, 32), ([90] * 20, [64] * 20, 4, 2, 128, 128)])
@pytest.mark.parametrize("vscale", [2.0 ** -16, 2.0 ** -60, 2.0 ** 14])
def test_log_sum_whatever_the_page_scales(h, lens, news, kv, group, d, page, vscale):
    """Sequences of one page, whose V has scales that are no powers of two and far from 1.
    They go into the exponents and out of the sums again: beyond the logits' error, lse
    has the roundings of values up to 2^5, 2^-19 in all (2^-17 where their exponents are
    up to 2^7)."""
    for seed in range(4):
        m = tc.Made(lens, kv, d, page, seed=seed, scales=(-12, -7))
        m.sV = vscale * (1 + torch.rand(m.sV.shape, generator=m.g))
        n = news or [1] * len(lens)
        q = tc.queries(m, sum(n), kv * group, seed=seed)
        O, L = tc.attend(h, m, q, news, scale=0.02)
        o, lse, mag, size = plain64.attention(plain64.value(m.K), m.sK, plain64.value(m.V), m.sV, m.table, m.kv_len, tc.starts_of(n), q, 0.02)
        assert ((O.double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -10 * mag).all()
        err = (L.double() - lse).abs()
        allowed = (2.0 ** -17 if vscale == 2.0 ** -60 else 2.0 ** -19) * (1 + size)
        assert (err <= allowed).all(), f"lse: worst {float((err / allowed).max())} of the tolerance"
