"""A decoder layer in 8 bits: a decoding step behind a prompt that the whole batch shares,
and a training step of its feed-forward block.

    python examples/decoder_layer_8bit.py

Decoding:
    x -> quantize -> QKV product -> norms of queries and keys with the rotation by
    positions -> append K, V -> attention behind the shared tokens -> quantize -> output
    product, then (with the residual) -> quantize -> gated pair of products, whose result
    is quantized in their epilogue -> down product
Training, of the block alone, with both passes in 8 bits:
    forward as above, with gate and up kept; dH from the down-projection's weight as it
    lies; the block's gradient as the operands of the products that give dX and the
    three weights' gradients

Both are compared with FP32.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_gemm_gb300 as mx  # noqa: E402

DEV = torch.device("cuda:0")


def _blocks(n):
    return -(-n // 128)


def quantize(x, block=mx.BLOCK_ROWS):
    """(codes, scales) of a matrix by rows, columns (stored transposed) or tiles."""
    r, c = x.shape
    shape, scales = {mx.BLOCK_ROWS: ((r, c), (r, _blocks(c))), mx.BLOCK_COLS: ((c, -(-r // 16) * 16), (c, _blocks(r))),
                     mx.BLOCK_TILES: ((r, c), (_blocks(r), _blocks(c)))}[block]
    out = torch.empty(shape, dtype=torch.uint8, device=DEV), torch.empty(scales, device=DEV)
    mx.mxgemm_quantize_block128(x, r, c, *out, block=block, stream=torch.cuda.current_stream())
    return out


class Handles:
    """One handle for weights as they lie out x in, one for the same contracted over their rows."""

    def __init__(self):
        self.nk, self.kn = mx.mxgemm_create(0), mx.mxgemm_create(0)
        mx.mxgemm_set_option(self.nk, mx.OPT_B_MAJOR, mx.B_N_BY_K)

    def product(self, a, b, m, n, k, dtype=torch.bfloat16, rows_k=False, b_block=128, into=None):
        """a . b^T (b n x k), or a . b (b k x n: rows_k); added to `into` where given."""
        c = torch.empty(m, n, dtype=dtype, device=DEV) if into is None else into
        mx.mxgemm_run_block128(self.kn if rows_k else self.nk, m, n, k, *a, *b, c, use_acc=into is not None,
                               out_dtype=mx.OUT_F32 if c.dtype is torch.float32 else mx.OUT_BF16, b_block=b_block,
                               stream=torch.cuda.current_stream())
        return c

    def gated(self, a, gate, up, m, n, k, keep=False):
        """Codes and scales of silu(a . gate^T) * (a . up^T), and both products where kept."""
        h = torch.empty(m, n, dtype=torch.uint8, device=DEV), torch.empty(m, _blocks(n), device=DEV)
        kept = [torch.empty(m, n, dtype=torch.bfloat16, device=DEV) if keep else None for _ in range(2)]
        mx.mxgemm_run_gated_block128(self.nk, m, n, k, *a, *gate, *up, h[0], H_scale=h[1], out_dtype=mx.OUT_E4M3, gate=kept[0], up=kept[1],
                                     stream=torch.cuda.current_stream())
        return h, *kept

    def close(self):
        for h in (self.nk, self.kn):
            status = mx.mxgemm_get_device_status(h)
            mx.mxgemm_destroy(h)
            if status[0] != mx.OK:
                raise RuntimeError(f"device status {status}")


def _weights(g, *shapes):
    return [(torch.randn(n, k, generator=g, device=DEV) * k ** -0.5).bfloat16() for n, k in shapes]


def _rotate(x, positions, freqs, interleaved):
    """The rotation in FP32 (angles in 64 bits)."""
    w = positions.double()[:, None] * freqs
    c, s = torch.cos(w).float()[:, None], torch.sin(w).float()[:, None]
    n, y = freqs.numel(), x.clone()
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., one], y[..., two] = x[..., one] * c - x[..., two] * s, x[..., two] * c + x[..., one] * s
    return y


def decode(batch=16, shared=1024, own=100, model=2048, heads=16, kv_heads=4, d=128, page=64, hidden=5632, rot=128, interleaved=False, seed=0):
    """Relative error of a decoding step's output against FP32: `batch` sequences of `own`
    tokens behind `shared` ones, of which the last is new."""
    if shared % page:
        raise ValueError("whole pages are shared")
    g = torch.Generator(device=DEV).manual_seed(seed)
    hd, kd, total = heads * d, kv_heads * d, shared + own
    w_qkv, w_out, w_gate, w_up, w_down = _weights(g, (hd + 2 * kd, model), (model, hd), (hidden, model), (hidden, model), (model, hidden))
    norm_q, norm_k = (1 + 0.1 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    freqs = mx.mxgemm_rope_frequencies(rot, 10000.0, mx.ROPE_BY_PARTS, 4.0, trained=4096).to(DEV)
    prompt = torch.randn(shared, model, generator=g, device=DEV).bfloat16()
    x = torch.randn(batch, own, model, generator=g, device=DEV).bfloat16()

    # ------------------------------------------------------------ in 8 bits
    hs = Handles()
    w8 = [quantize(w, mx.BLOCK_TILES) for w in (w_qkv, w_out, w_gate, w_up, w_down)]
    first, per = shared // page, -(-total // page) - shared // page
    pages = first + batch * per
    cache = mx.Cache(*(torch.zeros(pages, kv_heads, page, d, dtype=torch.uint8, device=DEV) for _ in range(2)),
                     *(torch.ones(pages, kv_heads, device=DEV) for _ in range(2)))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.cat([order[:first].expand(batch, first), order[first:].view(batch, per)], 1).contiguous()

    def heads_of(rows, positions):
        """Rotated queries and keys, and the values, of tokens."""
        t, stream = rows.shape[0], torch.cuda.current_stream()
        qkv = hs.product(quantize(rows), w8[0], t, hd + 2 * kd, model)
        q, k, v = qkv[:, :hd].view(t, heads, d), qkv[:, hd:hd + kd].view(t, kv_heads, d), qkv[:, hd + kd:].view(t, kv_heads, d)
        mx.mxgemm_norm_rope(q, k, q, k, positions=positions, freqs=freqs, interleaved=interleaved, q_weight=norm_q, k_weight=norm_k, stream=stream)
        return q, k, v

    def ints(*values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    stream = torch.cuda.current_stream()
    _, k, v = heads_of(prompt, torch.arange(shared, dtype=torch.int32, device=DEV))
    mx.mxgemm_cache_append(hs.nk, cache, table[:1, :max(1, -(-shared // page))].contiguous(), ints(shared), k, v, q_start=ints(0, shared), stream=stream)
    before = own - 1
    _, k, v = heads_of(x[:, :before].reshape(-1, model), (shared + torch.arange(before, dtype=torch.int32, device=DEV)).repeat(batch))
    lens = torch.full((batch,), total - 1, dtype=torch.int32, device=DEV)
    mx.mxgemm_cache_append(hs.nk, cache, table, lens, k, v, q_start=torch.arange(batch + 1, dtype=torch.int32, device=DEV) * before, stream=stream)
    token = x[:, -1].contiguous()
    q, k, v = heads_of(token, torch.full((batch,), total - 1, dtype=torch.int32, device=DEV))
    lens += 1
    mx.mxgemm_cache_append(hs.nk, cache, table, lens, k, v, stream=stream)
    o = torch.empty(batch, heads, d, dtype=torch.bfloat16, device=DEV)
    mx.mxgemm_cache_attention_shared(hs.nk, cache, table, lens, shared, q, o, stream=stream)
    y = hs.product(quantize(o.view(batch, hd)), w8[1], batch, model, hd) + token
    h, _, _ = hs.gated(quantize(y), w8[2], w8[3], batch, hidden, model)
    y = y + hs.product(h, w8[4], batch, model, hidden)
    hs.close()

    # ------------------------------------------------------------ in FP32
    def project(rows, positions):
        qkv = rows.float() @ w_qkv.float().t()
        t = rows.shape[0]
        q, k, v = qkv[:, :hd].view(t, heads, d), qkv[:, hd:hd + kd].view(t, kv_heads, d), qkv[:, hd + kd:].view(t, kv_heads, d)
        q, k = (_rotate(z * torch.rsqrt(z.square().mean(2, keepdim=True) + 1e-6) * n, positions, freqs, interleaved)
                for z, n in ((q, norm_q), (k, norm_k)))
        return q, k, v

    want = []
    for b in range(batch):
        q, k, v = project(torch.cat([prompt, x[b]]), torch.arange(total, device=DEV))
        q = q[-1].view(kv_heads, heads // kv_heads, d)
        p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * d ** -0.5, 2)
        z = torch.einsum("hgt,thd->hgd", p, v).reshape(1, hd) @ w_out.float().t() + x[b, -1].float()
        want.append(z + (torch.nn.functional.silu(z @ w_gate.float().t()) * (z @ w_up.float().t())) @ w_down.float().t())
    want = torch.cat(want)
    return float((y.float() - want).norm() / want.norm())


def train(tokens=4096, model=2048, hidden=5632, seed=0):
    """Relative errors of the feed-forward block's output and gradients against FP32."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w_gate, w_up, w_down = _weights(g, (hidden, model), (hidden, model), (model, hidden))
    x = torch.randn(tokens, model, generator=g, device=DEV).bfloat16()
    dy = (torch.randn(tokens, model, generator=g, device=DEV) * 0.01).bfloat16()
    hs = Handles()
    g8, u8, d8 = (quantize(w, mx.BLOCK_TILES) for w in (w_gate, w_up, w_down))
    tall = -(-tokens // 16) * 16

    h, gate, up = hs.gated(quantize(x), g8, u8, tokens, hidden, model, keep=True)
    y = hs.product(h, d8, tokens, model, hidden)

    dh = hs.product(quantize(dy), d8, tokens, hidden, model, rows_k=True)
    rows = {n: (torch.empty(tokens, hidden, dtype=torch.uint8, device=DEV), torch.empty(tokens, _blocks(hidden), device=DEV))
            for n in ("dgate_rows", "dup_rows")}
    cols = {n: (torch.empty(hidden, tall, dtype=torch.uint8, device=DEV), torch.empty(hidden, _blocks(tokens), device=DEV))
            for n in ("dgate_cols", "dup_cols", "hidden_cols")}
    mx.mxgemm_gated_backward(gate, up, dh, tokens, hidden, stream=torch.cuda.current_stream(), **rows, **cols)
    dx = hs.product(rows["dgate_rows"], g8, tokens, model, hidden, torch.float32, rows_k=True)
    hs.product(rows["dup_rows"], u8, tokens, model, hidden, rows_k=True, into=dx)
    x_cols, dy_cols = quantize(x, mx.BLOCK_COLS), quantize(dy, mx.BLOCK_COLS)
    d_gate = hs.product(cols["dgate_cols"], x_cols, hidden, model, tall, torch.float32, b_block=1)
    d_up = hs.product(cols["dup_cols"], x_cols, hidden, model, tall, torch.float32, b_block=1)
    d_down = hs.product(dy_cols, cols["hidden_cols"], model, hidden, tall, torch.float32, b_block=1)
    hs.close()

    leaves = [t.float().requires_grad_() for t in (x, w_gate, w_up, w_down)]
    xf, gf, uf, df = leaves
    out = (torch.nn.functional.silu(xf @ gf.t()) * (xf @ uf.t())) @ df.t()
    wants = torch.autograd.grad(out, leaves, dy.float())
    found = dict(zip(("y", "dx", "dgate", "dup", "ddown"), zip((y, dx, d_gate, d_up, d_down), (out.detach(), *wants))))
    return {n: float((a.float() - b).norm() / b.norm()) for n, (a, b) in found.items()}


if __name__ == "__main__":
    print(f"decoding step behind a shared prompt against FP32: relative error {decode():.4f}")
    print("feed-forward block's training step against FP32:", ", ".join(f"{n} {e:.4f}" for n, e in train().items()))
