"""Captured calls and a workspace that grows afterwards: a graph keeps the block
that it was captured with, and a call that is captured first needs none before."""
import ctypes

import pytest
import torch

import test_gpu_block128 as tb
import test_gpu_cache as tc

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_gemm_gb300")
DEV = "cuda:0"


@pytest.fixture
def h():
    h = mx.mxgemm_create(0)
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
    yield h
    mx.mxgemm_destroy(h)


class Step:
    """A decoding attention whose keys are split over CTAs, and a product whose K is."""

    def __init__(self, h):
        self.h = h
        m = self.m = tc.Made([9000, 700], 2, 128, 64)
        self.cache, self.table = m.cache(), m.table_tensor()
        self.lens = torch.tensor(m.kv_len, dtype=torch.int32, device=DEV)
        self.q = tc.queries(m, 2, 16).to(DEV)
        self.O = torch.empty_like(self.q)
        self.ops = [t.to(DEV) for t in tb.operands(300, 300, 4096, 128, 1)]
        self.C = torch.empty(300, 300, device=DEV)

    def __call__(self):
        s = torch.cuda.current_stream()
        mx.mxgemm_cache_attention(self.h, self.cache, self.table, self.lens, self.q, self.O, stream=s)
        mx.mxgemm_run_block128(self.h, 300, 300, 4096, *self.ops, self.C, stream=s)

    def results(self):
        torch.cuda.synchronize()
        return self.O.clone(), self.C.clone()

    def clear(self):
        self.O.zero_()
        self.C.zero_()


def grow(h):
    """Calls that need far more workspace: a prompt's parts, and the MX product's re-pitched B."""
    m = tc.Made([6000], 1, 128, 64)
    tc.attend(h, m, tc.queries(m, 2000, 1), [2000])
    K, N = 8192, 8008
    A, B = (torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (256 * K, K * N))
    As, Bs = (torch.full((n,), 127, dtype=torch.uint8, device=DEV) for n in (256 * K // 32, N * K // 32))
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_K_BY_N)
    mx.mxgemm_run(h, 256, N, K, A, As, B, Bs, torch.empty(256, N, device=DEV))
    mx.mxgemm_set_option(h, mx.OPT_B_MAJOR, mx.B_N_BY_K)
    torch.cuda.synchronize()


@pytest.mark.parametrize("before", [True, False])
def test_replay_after_growth(h, before):
    """`before`: an eager call of the sizes comes first."""
    other = mx.mxgemm_create(0)
    mx.mxgemm_set_option(other, mx.OPT_B_MAJOR, mx.B_N_BY_K)
    eager = Step(other)
    eager()
    want = eager.results()
    step = Step(h)
    if before:
        step()
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        step.clear()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(step.results(), want))
        grow(h)
        grow(other)  # takes what was freed, if anything was
    step.clear()
    step()
    assert all(torch.equal(a, b) for a, b in zip(step.results(), want))
    second = torch.cuda.CUDAGraph()  # with the grown workspace
    with torch.cuda.graph(second):
        step()
    for g in (second, graph):
        step.clear()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(step.results(), want))
    assert mx.mxgemm_get_device_status(h) == (0, 0) and mx.mxgemm_get_device_status(other) == (0, 0)
    del graph, second
    mx.mxgemm_destroy(other)


def test_mx_product_captured_before_growth(h):
    """The same for the MX product, whose repacked scales lie in the workspace; its
    plan is made by an eager call."""
    g = torch.Generator().manual_seed(3)
    M, N, K = 300, 512, 1024
    A, B = tb.random_codes((M, K), g).to(DEV), tb.random_codes((N, K), g).to(DEV)
    As, Bs = (torch.randint(120, 134, (n, K // 32), generator=g, dtype=torch.uint8).to(DEV) for n in (M, N))
    C = torch.empty(M, N, device=DEV)
    call = lambda: mx.mxgemm_run(h, M, N, K, A, As, B, Bs, C, stream=torch.cuda.current_stream())
    call()
    torch.cuda.synchronize()
    want = C.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)
        grow(h)
    del graph


def node_types(call):
    """cudaGraphNodeType of each node that `call` adds to a capture (kernel 0, memset 2)."""
    rt = ctypes.CDLL("libcudart.so.13")
    s = torch.cuda.Stream()
    graph, n = ctypes.c_void_p(), ctypes.c_size_t(0)
    with torch.cuda.stream(s):
        assert rt.cudaStreamBeginCapture(ctypes.c_void_p(s.cuda_stream), 1) == 0
        call()
        assert rt.cudaStreamEndCapture(ctypes.c_void_p(s.cuda_stream), ctypes.byref(graph)) == 0
    assert rt.cudaGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes, kind = (ctypes.c_void_p * n.value)(), ctypes.c_int()
    assert rt.cudaGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    kinds = []
    for node in nodes:
        assert rt.cudaGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kinds.append(kind.value)
    assert rt.cudaGraphDestroy(graph) == 0
    return kinds


@pytest.mark.parametrize("packed", [False, True])
def test_mx_product_with_shared_tiles_is_replayed(h, packed):
    """Tiles that several CTAs share: a replay waits for its own partial sums, not for
    the last replay's, which came of other inputs."""
    g = torch.Generator().manual_seed(4)
    M, N, K = 2560, 2560, 8192  # 100 tiles of 256 x 256, 64 K steps
    mx.mxgemm_set_option(h, mx.OPT_SCALE_LAYOUT, mx.SCALES_PACKED if packed else mx.SCALES_ROW_MAJOR)
    sources = [tb.random_codes((M, K), g).to(DEV) for _ in range(3)]
    A, B = sources[0].clone(), tb.random_codes((N, K), g).to(DEV)
    n = M * K // 32 if not packed else mx.mxgemm_scale_bytes(M, K, False, mx.SCALES_PACKED)
    As, Bs = (torch.randint(124, 130, (n,), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2))
    C = torch.empty(M, N, device=DEV)
    call = lambda: mx.mxgemm_run(h, M, N, K, A, As, B, Bs, C, stream=torch.cuda.current_stream())
    want = []
    for a in sources:
        A.copy_(a)
        call()
        torch.cuda.synchronize()
        want.append(C.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    assert 2 in node_types(call)  # the flags of the shared tiles are cleared by every replay
    for i in (0, 1, 2, 1, 0, 2, 0):
        A.copy_(sources[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want[i])
        if i == 2:
            call()
            torch.cuda.synchronize()
            assert torch.equal(C, want[i])
    assert mx.mxgemm_get_device_status(h) == (0, 0)
