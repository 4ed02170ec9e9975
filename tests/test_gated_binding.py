"""What the binding of the gated products and their gradient refuses, without a GPU:
tensors whose plain addresses would be read as something else."""
import pytest
import torch

mx = pytest.importorskip("block_scaled_gemm_gb300")

M, N, K = 20, 144, 272
KB, NB = 3, 2


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def run_args():
    return dict(A=codes(M, K), A_scale=torch.zeros(M, KB), G=codes(N, K), G_scale=torch.zeros(NB, KB), U=codes(K, N), U_scale=torch.zeros(KB, NB),
                H=codes(M, N), H_scale=torch.zeros(M, NB), gate=torch.zeros(M, N, dtype=torch.bfloat16), up=torch.zeros(M, N, dtype=torch.bfloat16))


def run(out_dtype=None, **kw):
    return mx.mxgemm_run_gated_block128(None, M, N, K, **{**run_args(), **kw}, out_dtype=mx.OUT_E4M3 if out_dtype is None else out_dtype, check=False)


def test_run_takes_what_is_right():
    assert run() == mx.ERR_INVALID_VALUE  # no handle
    assert run(A=codes(M, K).view(torch.float8_e4m3fn), G=codes(N * K), H=codes(2 * M, N)) == mx.ERR_INVALID_VALUE
    assert run(H=torch.zeros(M, N), H_scale=None, out_dtype=mx.OUT_F32) == mx.ERR_INVALID_VALUE
    assert run(**{k: v.data_ptr() for k, v in run_args().items()}) == mx.ERR_INVALID_VALUE
    assert run(**{k: None for k in run_args()}) == mx.ERR_INVALID_VALUE


@pytest.mark.parametrize("name", list(run_args()))
def test_run_refuses(name):
    t = run_args()[name]
    wide = torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)
    for bad in (t.double(), t.half(), wide[:, :t.shape[1]], wide[:, ::2], t[:-1], torch.zeros(t.shape[1], t.shape[0], dtype=t.dtype).t()):
        with pytest.raises(ValueError, match=name):
            run(**{name: bad})


def test_run_refuses_types_of_h():
    for out, dtype in ((mx.OUT_BF16, torch.float16), (mx.OUT_BF16, torch.int16), (mx.OUT_F32, torch.int32), (mx.OUT_F32, torch.float64)):
        with pytest.raises(ValueError, match="H"):
            run(H=torch.zeros(M, N, dtype=dtype), H_scale=None, out_dtype=out)


R, C = 20, 144


def grad_args():
    b = torch.zeros(R, C, dtype=torch.bfloat16)
    rows, cols = (codes(R, C), torch.zeros(R, 2)), (codes(C, 32), torch.zeros(C, 1))
    return dict(gate=b, up=b, dH=b, dgate=b, dup=b, dgate_rows=rows, dup_rows=rows, dgate_cols=cols, dup_cols=cols, hidden_cols=cols)


def grad(**kw):
    return mx.mxgemm_gated_backward(**{**grad_args(), **kw}, R=R, C=C, check=False)


def test_gradient_takes_what_is_right():
    ok = (mx.ERR_INVALID_VALUE, mx.ERR_CUDA)  # host memory
    assert grad() in ok and grad(dH=torch.zeros(R, C)) in ok
    assert grad(dH=torch.zeros(R, C).data_ptr(), x_dtype=mx.IN_F32) in ok
    assert grad(hidden_cols=None, dgate=None) in ok


@pytest.mark.parametrize("name", list(grad_args()))
def test_gradient_refuses(name):
    given = grad_args()[name]
    for i in range(2 if isinstance(given, tuple) else 1):
        t = given[i] if isinstance(given, tuple) else given
        wide = torch.zeros(t.shape[0], 2 * t.shape[1] + 2, dtype=t.dtype)
        bads = [t.double(), t.half(), t[:-1], wide[:, ::2][:, :t.shape[1]], wide[:, :t.shape[1]]]
        for bad in bads:
            if bad.is_contiguous() and bad.dtype == t.dtype and bad.numel() >= t.numel():
                continue  # (one column: dense all the same)
            with pytest.raises(ValueError):
                grad(**{name: (bad, given[1]) if i == 0 and isinstance(given, tuple) else (given[0], bad) if isinstance(given, tuple) else bad})


def test_gradients_dh_is_what_x_dtype_says():
    with pytest.raises(ValueError, match="dH"):
        grad(x_dtype=mx.IN_F32)
    with pytest.raises(ValueError, match="dH"):
        grad(dH=torch.zeros(R, C), x_dtype=mx.IN_BF16)
