"""One attention layer in 8 bits, prompt and then token by token.

    python examples/attention_layer_8bit.py

Both projections multiply E4M3 operands with one scale per block of 128, and
the keys and values stay in an 8-bit paged cache:

    x -> quantize -> QKV product -> append K, V -> attention -> quantize -> output product

The result is compared with the same layer in FP32 (weights, activations and
cache unrounded), and a decoding step is timed.
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


class Weight8:
    """A linear layer's weight (out x in) in E4M3, one scale per 128 x 128."""

    def __init__(self, w, stream=None):
        self.n, self.k = w.shape
        self.codes = torch.empty(self.n, self.k, dtype=torch.uint8, device=w.device)
        self.scales = torch.empty(_blocks(self.n), _blocks(self.k), device=w.device)
        mx.mxgemm_quantize_block128(w, self.n, self.k, self.codes, self.scales, block=mx.BLOCK_TILES, stream=stream)


class AttentionLayer8:
    """Grouped-query attention with 8-bit projections and cache."""

    def __init__(self, w_qkv, w_out, heads, kv_heads, head_dim, pages, page_size, max_tokens):
        self.heads, self.kv, self.d = heads, kv_heads, head_dim
        self.w_qkv, self.w_out = Weight8(w_qkv), Weight8(w_out)
        self.h = mx.mxgemm_create(0)
        mx.mxgemm_set_option(self.h, mx.OPT_B_MAJOR, mx.B_N_BY_K)  # weights as they lie, out x in
        codes = [torch.zeros(pages, kv_heads, page_size, head_dim, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.ones(pages, kv_heads, device=DEV) for _ in range(2)]
        self.cache = mx.Cache(*codes, *scales)
        width = max(w_qkv.shape[1], w_out.shape[1])
        self.codes = torch.empty(max_tokens * width, dtype=torch.uint8, device=DEV)
        self.scales = torch.empty(max_tokens * _blocks(width), device=DEV)

    def project(self, x, w, out, stream):
        """out = x . w^T with x quantized by rows."""
        t, k = x.shape
        mx.mxgemm_quantize_block128(x, t, k, self.codes, self.scales, block=mx.BLOCK_ROWS, stream=stream)
        mx.mxgemm_run_block128(self.h, t, w.n, k, self.codes, self.scales, w.codes, w.scales, out,
                               out_dtype=mx.OUT_BF16, stream=stream)

    def __call__(self, x, page_table, kv_len, q_start=None, stream=None):
        """x: tokens x model dim, bfloat16; kv_len: lengths with these tokens."""
        stream = stream or torch.cuda.current_stream()
        t, hd, kd = x.shape[0], self.heads * self.d, self.kv * self.d
        qkv = torch.empty(t, self.w_qkv.n, dtype=torch.bfloat16, device=DEV)
        self.project(x, self.w_qkv, qkv, stream)
        q = qkv[:, :hd].view(t, self.heads, self.d)
        k, v = (qkv[:, hd + i * kd:hd + (i + 1) * kd].view(t, self.kv, self.d) for i in (0, 1))
        mx.mxgemm_cache_append(self.h, self.cache, page_table, kv_len, k, v, q_start=q_start, stream=stream)
        o = torch.empty(t, self.heads, self.d, dtype=torch.bfloat16, device=DEV)
        mx.mxgemm_cache_attention(self.h, self.cache, page_table, kv_len, q, o, q_start=q_start, stream=stream)
        y = torch.empty(t, self.w_out.n, dtype=torch.bfloat16, device=DEV)
        self.project(o.view(t, hd), self.w_out, y, stream)
        return y

    def status(self):
        return mx.mxgemm_get_device_status(self.h)

    def close(self):
        mx.mxgemm_destroy(self.h)


def layer_fp32(x, w_qkv, w_out, heads, kv_heads, d):
    """The layer on one whole sequence in FP32."""
    t = x.shape[0]
    qkv = x.float() @ w_qkv.float().t()
    hd, kd = heads * d, kv_heads * d
    q = qkv[:, :hd].view(t, heads, d).transpose(0, 1)
    k, v = (qkv[:, hd + i * kd:hd + (i + 1) * kd].view(t, kv_heads, d).transpose(0, 1).repeat_interleave(heads // kv_heads, 0)
            for i in (0, 1))
    s = (q @ k.transpose(1, 2)) * d ** -0.5
    s = s.masked_fill(torch.ones(t, t, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    return (torch.softmax(s, 2) @ v).transpose(0, 1).reshape(t, hd) @ w_out.float().t()


def run(batch=8, prompt=600, steps=4, model=2048, heads=16, kv_heads=4, d=128, page=64, seed=0):
    """(relative error of all outputs against FP32, seconds of a decoding step)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    w_qkv = (randn((heads + 2 * kv_heads) * d, model) * model ** -0.5).bfloat16()
    w_out = (randn(model, heads * d) * (heads * d) ** -0.5).bfloat16()
    x = randn(batch, prompt + steps, model).bfloat16()
    width = -(-(prompt + steps) // page)
    layer = AttentionLayer8(w_qkv, w_out, heads, kv_heads, d, batch * width, page, batch * prompt)
    table = torch.randperm(batch * width, generator=g, device=DEV).to(torch.int32).view(batch, width)
    starts = torch.arange(batch + 1, dtype=torch.int32, device=DEV) * prompt
    lens = torch.full((batch,), prompt, dtype=torch.int32, device=DEV)
    y = [layer(x[:, :prompt].reshape(batch * prompt, model), table, lens, starts).view(batch, prompt, model)]
    for i in range(steps):
        lens += 1
        y.append(layer(x[:, prompt + i].contiguous(), table, lens)[:, None])
    y = torch.cat(y, 1).float()
    want = torch.stack([layer_fp32(x[b], w_qkv, w_out, heads, kv_heads, d) for b in range(batch)])
    error = float((y - want).norm() / want.norm())
    token = x[:, -1].contiguous()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(23):  # the last token again and again: the same positions are written
        if i == 3:
            a.record()
        layer(token, table, lens)
    b.record()
    torch.cuda.synchronize()
    status = layer.status()
    layer.close()
    if status[0] != mx.OK:
        raise RuntimeError(f"device status {status}")
    return error, a.elapsed_time(b) / 20e3


if __name__ == "__main__":
    err, step = run()
    print(f"8-bit layer against FP32: relative error {err:.4f}; a decoding step of 8 sequences {step * 1e6:.0f} us (as calls)")
