"""Plain 64-bit implementations of the block-128 product, its quantizer and the
8-bit cache's append and attention, from their definitions; the tests' side."""
from __future__ import annotations

import math

import torch


def value(codes: torch.Tensor) -> torch.Tensor:
    """E4M3 codes -> float64, by the format (bias 7, subnormals, 0x7F NaN)."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(torch.tensor(2.0, dtype=torch.float64), (e - 10).double()))
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def value_e5m2(codes: torch.Tensor) -> torch.Tensor:
    """Finite E5M2 codes -> float64 (bias 15)."""
    c = codes.to(torch.int64)
    e, m = (c >> 2) & 31, (c & 3).double()
    v = torch.where(e == 0, m * 2.0 ** -16, (4 + m) * torch.pow(torch.tensor(2.0, dtype=torch.float64), (e - 17).double()))
    return torch.where(c >= 128, -v, v)


def e4m3(y: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 value, ties to even, saturating."""
    y = y.double().clamp(-448, 448)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), torch.frexp(y)[1].clamp(min=-5).double() - 4)
    return torch.round(y / step) * step


def spread(scale: torch.Tensor, dim: int, n: int) -> torch.Tensor:
    """Scales of blocks of 128 along dim, one for each of n elements."""
    return scale.double().repeat_interleave(128, dim).narrow(dim, 0, n)


def product(a, sa, b, sb, b_block):
    """(C, sum of |terms|) for a M x K, b N x K float64 and their scales."""
    k, n = a.shape[1], b.shape[0]
    a = a * spread(sa, 1, k)
    sb = spread(sb, 1, k)
    b = b * (sb if b_block == 1 else sb.repeat_interleave(128, 0)[:n])
    return a @ b.t(), a.abs() @ b.abs().t()


def quantize(x, block):
    """(code values, scales) in 64 bits but for the FP32 steps that the definition fixes."""
    x = x.float()
    r, c = x.shape
    br, bc = {"rows": (1, 128), "cols": (128, 1), "tiles": (128, 128)}[block]
    pad = torch.nn.functional.pad(x, (0, -c % bc, 0, -r % br))
    nb = pad.view(pad.shape[0] // br, br, pad.shape[1] // bc, bc)
    top = nb.abs().amax((1, 3)).clamp(min=2.0 ** -100)
    inv = (torch.full_like(top, 448.0) / top).repeat_interleave(br, 0)[:r].repeat_interleave(bc, 1)[:, :c]
    codes, scales = e4m3(x * inv), top / 448.0
    if block == "cols":
        codes, scales = torch.nn.functional.pad(codes.t(), (0, -r % 16)), scales.t()
    return codes, scales


def need(amax: float) -> float:
    """Least power of two >= amax / 448, 2^-64 at least."""
    p = 2.0 ** -64
    while p * 448 < amax:
        p *= 2
    return p


def append(values, scale, table, kv_len, starts, x):
    """One of K and V: values (pages, heads, page, d) float64 of the codes and
    scale, changed in place."""
    page = values.shape[2]
    for b, t in enumerate(kv_len):
        n = starts[b + 1] - starts[b]
        first = t - n
        for p in range(first // page, -(-t // page)) if n else ():
            lo, hi, pg = max(p * page, first), min((p + 1) * page, t), table[b][p]
            y = x[starts[b] + lo - first:starts[b] + hi - first].double()
            for h in range(values.shape[1]):
                s = need(float(y[:, h].abs().max()))
                k = lo - p * page
                if k:
                    s = max(s, float(scale[pg, h]))
                    values[pg, h, :k] = e4m3(values[pg, h, :k] * (float(scale[pg, h]) / s))
                values[pg, h, k:hi - p * page] = e4m3(y[:, h] / s)
                scale[pg, h] = s


def attention(values_k, sk, values_v, sv, table, kv_len, starts, q, scale, causal=True, window=0, sinks=0):
    """(o, lse, sum of p |v|, largest sum of |scale q k|) per token and head."""
    page, kv = values_k.shape[2], values_k.shape[1]
    tokens, heads, d = q.shape
    o = torch.zeros(tokens, heads, d, dtype=torch.float64)
    mag = torch.zeros_like(o)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    size = torch.zeros(tokens, heads, dtype=torch.float64)
    for b, t in enumerate(kv_len):
        n = starts[b + 1] - starts[b]
        if t == 0 or n == 0:
            continue
        pages = table[b][:-(-t // page)]
        pos = torch.arange(t - n, t)[:, None]
        j = torch.arange(t)[None]
        seen = (j <= pos) if causal else torch.ones(n, t, dtype=torch.bool)
        if window:
            seen = seen & ((pos - j < window) | (j < sinks))
        absent = torch.tensor([p < 0 or p >= values_k.shape[0] for p in pages]).repeat_interleave(page)[:t]
        seen = seen & ~absent[None]
        at = torch.tensor([p if 0 <= p < values_k.shape[0] else 0 for p in pages])
        for i in range(kv):
            k = (values_k[at, i] * sk[at, i].double()[:, None, None]).reshape(-1, d)[:t]
            v = (values_v[at, i] * sv[at, i].double()[:, None, None]).reshape(-1, d)[:t]
            some = seen.any(0)
            k, v = torch.where(some[:, None], k, 0.0), torch.where(some[:, None], v, 0.0)
            for h in range(i * (heads // kv), (i + 1) * (heads // kv)):
                x = q[starts[b]:starts[b + 1], h].double()
                s = (x @ k.t() * scale).masked_fill(~seen, -math.inf)
                top = s.amax(1, keepdim=True).clamp(min=-1e300)
                w = torch.exp(s - top)
                l = w.sum(1, keepdim=True)
                p = w / torch.where(l > 0, l, 1.0)
                o[starts[b]:starts[b + 1], h] = p @ v
                mag[starts[b]:starts[b + 1], h] = p @ v.abs()
                lse[starts[b]:starts[b + 1], h] = (top + torch.log(l))[:, 0]
                size[starts[b]:starts[b + 1], h] = (abs(scale) * (x.abs() @ k.abs().t())).masked_fill(~seen, 0).amax(1)
    return o, lse, mag, size
