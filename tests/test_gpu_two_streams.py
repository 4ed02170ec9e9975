"""Two handles on two streams at once: work that is split over CTAs has no CTA that waits
for another, so that calls that share the SMs end as they would alone, bit for bit."""
import pytest
import torch

import test_gpu_block128 as tb
import test_gpu_cache as tc

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"


class Program:
    """Products whose tiles are cut along K (alone and after whole ones), split single
    tokens, and prompts whose keys are cut, into outputs of their own."""

    def __init__(self, seed):
        self.h = mx.mxgemm_create(0)
        mx.mxgemm_set_option(self.h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
        self.products = []
        for m, n, k, b_block in ((300, 300, 4096, 128), (2600, 2304, 4096, 1), (20, 1000, 4096, 128)):
            ops = [t.to(DEV) for t in tb.operands(m, n, k, b_block, seed + m)]
            self.products.append((m, n, k, b_block, ops, torch.empty(m, n, device=DEV)))
        self.attentions = []
        for lens, news, kv, group in (([9000, 700], None, 2, 8), ([5000], [70], 1, 1), ([1900, 700, 64], [70, 64, 66], 60, 1)):
            m = tc.Made(lens, kv, 128, 64, seed=seed)
            n = news or [1] * len(lens)
            q = tc.queries(m, sum(n), kv * group, seed=seed).to(DEV)
            starts = None if news is None else torch.tensor(tc.starts_of(news), dtype=torch.int32, device=DEV)
            self.attentions.append((m.cache(), m.table_tensor(), torch.tensor(lens, dtype=torch.int32, device=DEV), q, torch.empty_like(q), starts))

    def __call__(self, stream):
        for m, n, k, b_block, ops, C in self.products:
            mx.mxgemm_run_block128(self.h, m, n, k, *ops, C, b_block=b_block, stream=stream)
        for cache, table, lens, q, O, starts in self.attentions:
            mx.mxgemm_cache_attention(self.h, cache, table, lens, q, O, q_start=starts, stream=stream)

    def results(self):
        return [p[-1] for p in self.products] + [a[4] for a in self.attentions]


def test_equal_bits_side_by_side():
    programs = [Program(1), Program(2)]
    streams = [torch.cuda.Stream() for _ in programs]
    try:
        want = []
        for p in programs:
            p(torch.cuda.current_stream())
            torch.cuda.synchronize()
            want.append([t.clone() for t in p.results()])
        for _ in range(10):
            for p in programs:
                for t in p.results():
                    t.zero_()
            torch.cuda.synchronize()
            for _ in range(5):
                for p, s in zip(programs, streams):
                    p(s)
            torch.cuda.synchronize()
            for p, w in zip(programs, want):
                assert all(torch.equal(a, b) for a, b in zip(p.results(), w))
                assert mx.mxgemm_get_device_status(p.h) == (0, 0)
    finally:
        for p in programs:
            mx.mxgemm_destroy(p.h)
