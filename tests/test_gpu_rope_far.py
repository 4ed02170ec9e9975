"""The rotation at far positions with frequencies as they are (none a fraction of a turn):
angles are within 2^-24 of half a turn whatever the position and the frequency.

The reference reduces position * frequency by 2 pi in whole numbers of 256 bits.
Tolerance, of the sizes of a pair: the angle's 2^-24 of half a turn (2^-22.3), sine and
cosine 2^-23 (two units in FP32's last place), a product with the factor and two
steps of a sum, 2^-24 each: 2^-21 in all."""
import math

import pytest
import torch

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"
BITS = 256


def inverse_arctangent(n):
    """atan(1 / n) times 2^BITS."""
    total, term, k = 0, (1 << BITS) // n, 0
    while term:
        total += (-1) ** k * (term // (2 * k + 1))
        term //= n * n
        k += 1
    return total


TWO_PI = 8 * (4 * inverse_arctangent(5) - inverse_arctangent(239))  # Machin's formula


def angle64(position, freq):
    """position * freq reduced to one turn, in 64 bits."""
    n, d = float(freq).as_integer_ratio()
    turns = ((position * n) << (2 * BITS)) // (d * TWO_PI)  # times 2^BITS
    return 2 * math.pi * ((turns % (1 << BITS)) / (1 << BITS))


def test_reference():
    for p, f in ((0, 1.0), (1, 1.0), (-3, 0.7), (100, 2.5), (12345, 1e-3), (7, 100.25)):
        a = angle64(p, f)
        assert abs(math.cos(a) - math.cos(p * f)) < 1e-11 and abs(math.sin(a) - math.sin(p * f)) < 1e-11
    assert TWO_PI / 2 ** BITS == 2 * math.pi


@pytest.mark.gpu
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("fastest", [1.0, 37.5, 1000.0, 2.0 ** 40])
def test_ordinary_frequencies(fastest, back):
    h = mx.mxgemm_create(0)
    freqs = mx.mxgemm_rope_frequencies(128) * fastest
    positions = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 2 ** 30 + 7, 123456789, -987654321, 1, -1, 0, 2 ** 28 - 1]
    g = torch.Generator().manual_seed(3)
    x = torch.randn(len(positions), 2, 128, generator=g)
    kw = {"positions": torch.tensor(positions, dtype=torch.int32, device=DEV), "freqs": freqs.to(DEV)}
    out = torch.empty(x.shape, device=DEV)
    if back:
        mx.mxgemm_norm_rope_backward(h, x.to(DEV), None, out, None, **kw)
    else:
        mx.mxgemm_norm_rope(x.to(DEV), None, out, None, **kw)
    w = torch.tensor([[angle64(p, f) for f in freqs.tolist()] for p in positions], dtype=torch.float64)[:, None] * (-1 if back else 1)
    a, b = x.double().split(64, 2)
    want = torch.cat((a * torch.cos(w) - b * torch.sin(w), b * torch.cos(w) + a * torch.sin(w)), 2)
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    worst = ((out.cpu().double() - want).abs() / size).max().item()
    assert worst <= 2.0 ** -21, f"{worst * 2 ** 21} of the tolerance"
    mx.mxgemm_destroy(h)
