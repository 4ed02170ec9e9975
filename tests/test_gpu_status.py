"""Reading a status word is ordered by the stream that is given, not by the
default one, which other streams need not wait for: the word's clearing comes
before whatever follows on that stream."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")


@pytest.mark.parametrize("handle", [True, False])
def test_read_does_not_wait_for_the_default_stream(handle):
    h = mx.mxgemm_create(0) if handle else None
    s = torch.cuda.Stream()
    read = (lambda: mx.mxgemm_get_device_status(h, s)) if handle else (lambda: mx.mxgemm_noalloc_get_status(s))
    read()
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    torch.cuda._sleep(1_000_000_000)  # about half a second on the default stream
    done.record()
    t0 = time.perf_counter()
    assert read() == (0, 0)
    waited, busy = time.perf_counter() - t0, not done.query()
    torch.cuda.synchronize()
    if handle:
        mx.mxgemm_destroy(h)
    assert busy and waited < 0.2
