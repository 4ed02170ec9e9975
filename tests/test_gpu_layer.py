"""The parts of a transformer layer together and at their ends: a decoder layer behind a
shared prompt and a training step of its feed-forward block (the example), calls of two
handles on two streams at once, and matrices whose offsets pass 32 bits."""
import importlib.util
import math
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    path = Path(__file__).resolve().parents[1] / "examples" / "decoder_layer_8bit.py"
    spec = importlib.util.spec_from_file_location("decoder_layer_8bit", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kw", [dict(batch=3, shared=256, own=40, model=512, heads=8, kv_heads=2, d=64, page=32, hidden=1024, rot=32, interleaved=True),
                                dict(batch=5, shared=128, own=70, model=1024, heads=16, kv_heads=4, d=128, page=16, hidden=1536, rot=128, interleaved=False)])
def test_decoder_layer(example, kw):
    """Each of the seven roundings to E4M3 (x, QKV weight, K or V, o, output weight; then
    the block's x, its three weights and H) is off by 0.027 of a value in root mean
    square; a path takes at most nine of them, sqrt(9) 0.027 = 0.081, twice that allowed."""
    assert example.decode(**kw) < 0.17


@pytest.mark.parametrize("kw", [dict(tokens=200, model=512, hidden=768), dict(tokens=333, model=384, hidden=1040), dict(tokens=40, model=256, hidden=512)])
def test_feed_forward_gradients(example, kw):
    """Every gradient against the block's in FP32 by autograd: an operand of its last
    product is rounded once (0.027), what it was made of up to four times before:
    under 0.1 of its norm, twice that allowed."""
    for name, error in example.train(**kw).items():
        assert error < 0.2, (name, error)


def test_two_handles_on_two_streams():
    """Gated products and norms' gradients of two handles at once: the bits of single calls."""
    from test_gpu_gated import Made
    from test_gpu_rope import Case
    hs = [mx.mxgemm_create(0) for _ in range(2)]
    for h in hs:
        mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
    made, case = Made(20, 1040, 2048, 1), Case(700, 8, 2, 128, 128, False, torch.bfloat16, True)
    want = made.run(hs[0], True, "silu", "e4m3", False)
    want_dx, want_dw = case.backward(hs[0])
    w = [t.to(DEV) for pair in made.w for t in pair]
    a, sa = made.a.to(DEV), made.sa.to(DEV)
    rows, x, kw = case.on_device()
    dy = [v.to(DEV) for v in case.dy]
    outs = [[(torch.zeros(20, 1040, dtype=torch.uint8, device=DEV), torch.zeros(20, 9, device=DEV), [torch.zeros_like(v) for v in dy],
              [torch.zeros(128, device=DEV) for _ in range(2)]) for _ in range(8)] for _ in hs]
    sides = [torch.cuda.Stream() for _ in hs]
    torch.cuda.synchronize()
    for i in range(8):
        for h, side, out in zip(hs, sides, outs):
            H, sH, dx, dw = out[i]
            mx.mxgemm_run_gated_block128(h, 20, 1040, 2048, a, sa, *w, H, H_scale=sH, out_dtype=mx.OUT_E4M3, stream=side)
            mx.mxgemm_norm_rope_backward(h, dy[0], dy[1], dx[0], dx[1], q=x[0], k=x[1], dq_weight=dw[0], dk_weight=dw[1], stream=side, **kw)
    torch.cuda.synchronize()
    for out in outs:
        for H, sH, dx, dw in out:
            assert torch.equal(H.cpu(), want[0]) and torch.equal(sH.cpu(), want[1])
            assert all(torch.equal(p, q) for p, q in zip(dx + dw, want_dx + want_dw))
    for h in hs:
        assert mx.mxgemm_get_device_status(h) == (0, 0)
        mx.mxgemm_destroy(h)


def test_heads_with_a_pitch_past_32_bits():
    """Rows 2^31 elements apart: the same as dense ones."""
    t, heads, d = 3, 2, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn(t, heads, d, generator=g).bfloat16().to(DEV)
    far = torch.empty((t - 1) * 2 ** 31 + heads * d, dtype=torch.bfloat16, device=DEV)
    view = far.as_strided((t, heads, d), (2 ** 31, d, 1))
    view.copy_(x)
    kw = dict(positions=torch.arange(t, dtype=torch.int32, device=DEV), freqs=mx.mxgemm_rope_frequencies(d).to(DEV), q_weight=torch.ones(d, device=DEV))
    want = torch.empty_like(x)
    mx.mxgemm_norm_rope(x, None, want, None, **kw)
    mx.mxgemm_norm_rope(view, None, view, None, **kw)
    torch.cuda.synchronize()
    assert torch.equal(view, want)


def test_gradient_of_more_than_2_31_values():
    r, c = 80000, 28672
    gate = torch.full((r, c), 0.5, dtype=torch.bfloat16, device=DEV)
    up, dh, d = torch.full_like(gate, 2.0), torch.full_like(gate, 0.25), torch.zeros_like(gate)
    dh[-1, -3:] = -8.0
    mx.mxgemm_gated_backward(gate, up, dh, r, c, dgate=d)
    torch.cuda.synchronize()
    p = 1 / (1 + math.exp(-0.5))
    slope = 2 * (p + 0.5 * p * (1 - p))
    assert abs(float(d[0, 0]) - 0.25 * slope) <= 2.0 ** -8 * 0.25 * slope
    assert ((d[-1, -3:].float() + 8 * slope).abs() <= 2.0 ** -8 * 8 * slope).all() and abs(float(d[-1, -4]) - 0.25 * slope) <= 2.0 ** -8 * 0.25 * slope
    codes, scales = torch.zeros(r, c, dtype=torch.uint8, device=DEV), torch.zeros(r, c // 128, device=DEV)
    cols, cscales = torch.zeros(c, r, dtype=torch.uint8, device=DEV), torch.zeros(c, r // 128, device=DEV)
    mx.mxgemm_gated_backward(gate, up, dh, r, c, dup_rows=(codes, scales), dup_cols=(cols, cscales))
    torch.cuda.synchronize()
    one, eight = 0.25 * 0.5 * p, 8 * 0.5 * p
    assert abs(float(scales[0, 0]) * 448 - one) <= 2.0 ** -18 * one and abs(float(scales[-1, -1]) * 448 - eight) <= 2.0 ** -18 * eight
    assert int(codes[-1, -1]) == 0xFE and int(codes[0, 0]) == 0x7E and int(cols[-1, -1]) == 0xFE and int(cols[0, 0]) == 0x7E  # -448, 448
    assert abs(float(cscales[-1, -1]) * 448 - eight) <= 2.0 ** -18 * eight and abs(float(cscales[-1, -2]) * 448 - one) <= 2.0 ** -18 * one
