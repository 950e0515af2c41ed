"""Captured products and the memory they use: a larger call on the stream
leaves a graph the workspace and the operand copies it was captured with, and
a product that is captured without a call before it allocates nothing and is
right all the same."""
import pytest

import workloads
from tests._gpu import TOL, assert_close, lib, oracle_full

pytestmark = pytest.mark.gpu


def _call(g, a, b, c, mode, s):
    M, K = a.shape
    g.check(g.gemm_f32_ex(a, b, c, M, b.shape[1], K, mode, 0, s))


@pytest.mark.parametrize("mode", ["tc3x", "ffma", "tc1x"])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("shape", [(1024, 512, 1024), (1001, 513, 777), (3000, 4096, 2000)])
def test_graph_keeps_its_memory(shape, first, mode):
    import torch
    g = lib()
    M, K, N = shape
    A, B = workloads.make_inputs(M, K, N, "uniform", 60)
    a, b = torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda()
    c = torch.empty((M, N), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g.check(g.gemm_f32_release())                     # buffers of earlier tests' streams
    if first:
        with torch.cuda.stream(s):
            _call(g, a, b, c, mode, s)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):           # torch gives its free memory back as it enters
        free = torch.cuda.mem_get_info()[0]
        _call(g, a, b, c, mode, s)
        used = free - torch.cuda.mem_get_info()[0]
    assert used < (1 << 23)                           # no buffer (a kernel's code may be loaded at its first launch)
    for m, k, n in ((3001, 4099, 5003), (4100, 8192, 4100)):   # odd strides: copies; last waves that are split
        big = torch.rand((m, k), device="cuda"), torch.rand((k, n), device="cuda"), torch.empty((m, n), device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            _call(g, *big, mode, s)
        torch.cuda.synchronize()
    torch.full((1 << 28,), float("nan"), device="cuda")
    want, size = oracle_full(A, B)
    for _ in range(2):
        c.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert g.gemm_f32_status(s) == (0, 0)
        assert_close(c.cpu().numpy(), want, size, TOL[mode], "graph %s/%s" % (shape, mode))
