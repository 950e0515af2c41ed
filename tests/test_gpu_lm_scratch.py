"""The scratch of the language-model operators: what it held before a call
does not matter."""
import ctypes

import pytest

from tests._gpu import lib
from tests.test_gpu_vocab_loss import _check, _exact, _inputs, _torch

pytestmark = pytest.mark.gpu


def _scratch(stream, nbytes):
    """Address of the library's scratch for calls on a stream, by its internal function."""
    from accelerator_row_major_gb300 import _binding
    f = _binding.lib()._ZN13gemm_f32_impl15acquire_scratchEiP11CUstream_stm
    f.argtypes, f.restype = [ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t], ctypes.c_void_p
    return f(0, stream, nbytes)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [9, 200, 600])
def test_a_scratch_that_holds_anything(rows, kind):
    """Memory that an allocation returns is not zero: every word of the scratch holds 3.0 before the call."""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(rows, 100, 1200, kind, rows)
    want = _exact(x, w, y, kind)
    one, threes = torch.ones((1, 1), device="cuda"), torch.full((1, 1 << 18), 3.0, device="cuda")
    for call in (g.vocab_loss, g.vocab_loss_grad):
        call(x, w, y)                                   # sizes it
        at = _scratch(0, 1 << 18)
        g.check(g.gemm_f32(one, threes, at, 1, 1 << 16, 1))
        _check(call(x, w, y), want)


def _both(g, x, w, y, rows):
    """Loss with gradients, and a norm with its gradient, of the first `rows` rows."""
    a = x[:rows]
    n, mean, rstd = g.layer_norm(a)
    return g.vocab_loss_grad(a, w, y[:rows]) + (n, mean, rstd) + g.layer_norm_grad(a, n, None, mean, rstd)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_graphs_of_several_sizes_and_larger_calls(kind):
    """Graphs captured on one stream, without a call before them, keep their scratch while calls of other sizes
    come and go on that stream, while it is released, and while other streams compute."""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(1500, 264, 3001, kind, 7)
    sizes = (40, 700, 1500, 300)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for rows in sizes:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = _both(g, x, w, y, rows)
        graphs.append((graph, out))
    big = _inputs(4096, 520, 9001, kind, 8)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        g.vocab_loss_grad(*big)
    torch.cuda.synchronize()
    assert g.gemm_f32_release() == 0
    for seed in (1, 2):
        x2, w2, y2 = _inputs(1500, 264, 3001, kind, seed)
        for t, t2 in ((x, x2), (w, w2), (y, y2)):
            t.copy_(t2)
        want = [_both(g, x, w, y, rows) for rows in sizes]
        _check(want[1], _exact(x[:700], w, y[:700], kind))
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()                            # beside calls on the stream of the capture
            with torch.cuda.stream(s):
                g.vocab_loss_grad(*big)
        torch.cuda.synchronize()
        for (_, out), expected in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, expected))
    assert g.gemm_f32_status(None) == (0, 0)


def test_scratch_of_destroyed_graphs_comes_back():
    """Capturing again and again does not take more memory each time."""
    torch, _ = _torch()
    g = lib()
    x, w, y = _inputs(2000, 136, 20000, "bf16", 3)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    free = []
    for _ in range(6):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.vocab_loss_grad(x, w, y)
        graph.replay()
        torch.cuda.synchronize()
        free.append(torch.cuda.mem_get_info()[0])
        del graph
        torch.cuda.synchronize()
    # each takes some 80 MB of scratch; torch's own pools may still settle in the first rounds
    assert free[2] - free[5] < (64 << 20)


def test_threads_on_one_stream():
    """Host threads whose calls of different sizes share a stream, and so its scratch."""
    import threading
    torch, _ = _torch()
    g = lib()
    cases = [_inputs(rows, width, vocab, kind, rows) for rows, width, vocab, kind in
             ((600, 136, 3001, "bf16"), (1100, 72, 5000, "f32"), (20, 260, 9000, "bf16"), (300, 513, 1200, "f32"))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [_both(g, *c, c[0].shape[0]) for c in cases]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(cases))

    def work(i):
        try:
            with torch.cuda.stream(s):
                start.wait()
                got = [_both(g, *cases[i], cases[i][0].shape[0]) for _ in range(40)]
                s.synchronize()
                for out in got:
                    assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
        except Exception as e:      # collected and re-raised in the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]
    assert g.gemm_f32_status(s) == (0, 0)


def test_outputs_belong_to_the_stream_that_is_given():
    """Memory that the current stream has freed but still writes to does not become an output of another stream's
    call."""
    torch, _ = _torch()
    g = lib()
    x, w, _ = _inputs(512, 1024, 8, "f32", 1)
    xt = x.t().contiguous()
    want, product = g.layer_norm(x)[0], g.matmul(x, xt)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g.layer_norm(x, stream=s)
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    late = torch.empty_like(x).fill_(7.0)             # some 25 ms from now
    del late
    y = g.layer_norm(x, stream=s)[0]
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    c = g.matmul(x, xt, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(c, product)


FIRST_CALL_IN_A_CAPTURE = """
import ctypes
import sys
sys.path.insert(0, %r)
import torch
import accelerator_row_major_gb300 as g
x = torch.randn(600, 9000, device="cuda")
w = torch.randn(500, 9000, device="cuda") / 100
y = torch.randint(0, 500, (600,), device="cuda")
torch.cuda.synchronize()
stream = torch.cuda.Stream()
if %r:
    handle = ctypes.c_void_p()
    assert ctypes.CDLL("libcuda.so.1").cuStreamCreate(ctypes.byref(handle), 0) == 0
    stream = torch.cuda.ExternalStream(handle.value)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=stream):
    a = g.vocab_loss_grad(x, w, y)
    n, mean, rstd = g.layer_norm(x)
    b = g.layer_norm_grad(x, n, None, mean, rstd)
graph.replay()
torch.cuda.synchronize()
n2, mean, rstd = g.layer_norm(x)
want = g.vocab_loss_grad(x, w, y) + (n2,) + g.layer_norm_grad(x, n2, None, mean, rstd)
assert all(torch.equal(p, q) for p, q in zip(a + (n,) + b, want))
assert g.gemm_f32_status(None) == (0, 0)
print("same")
"""


@pytest.mark.parametrize("legacy", [False, True])
def test_first_call_of_a_process_in_a_capture(legacy):
    """The library sets the device up in whatever call comes first; `legacy`: a capture of a stream that the legacy
    default stream waits for, which takes no work meanwhile."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE % (root, legacy)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stdout + run.stderr[-3000:]
