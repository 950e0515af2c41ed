"""The norms at a block's ends, checkpoints and weight gradients as programs
use them: in graphs, on several streams and threads, one after the other in a
training step."""
import threading

import pytest

from tests._gpu import lib

pytestmark = pytest.mark.gpu


def _step(g, s, w):
    """The end of a block, the next one's product, and everything back through both with checkpoints."""
    import torch
    y, h, stats = g.block_norm(s["branch"], s["residual"], s["weight"], s["bias"], **s["how"])
    kept_y, kept_h, kept_b = g.checkpoint(y), g.checkpoint(h), g.checkpoint(s["branch"])
    dw = g.weight_grad(w, kept_y)
    grads = g.block_norm_grad(s["dy"], s["dh"], kept_h, kept_b, stats, s["weight"], **s["how"])
    return [y, h, stats, kept_y.codes.view(torch.uint8), kept_y.exponents[:, :1], g.restore(kept_h), dw] + [v for v in grads if v is not None]


def _args(b, rows, kind, seed, width=520):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + 100)
    s = b.inputs(rows, width, kind, "f32", "layer", "channel", True, seed, (1.0, 0.5))
    return s, torch.randn(rows, 200, generator=gen, device="cuda").to(b.TYPES[kind])


def _refill(s, w, s2, w2):
    import torch
    for k, v in s.items():
        if torch.is_tensor(v):
            v.copy_(s2[k])
    for k, v in s["how"].items():
        if torch.is_tensor(v):
            v.copy_(s2["how"][k])
    w.copy_(w2)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_graphs_of_several_sizes_beside_calls(kind):
    """Graphs captured without a call before them, replayed on new inputs while other calls of other sizes run on the
    stream of the capture and the library's memory is released: the same bits as the calls give."""
    import torch
    from tests import _block as b
    g = lib()
    sizes = (40, 1500, 300)
    args = [_args(b, r, kind, r) for r in sizes]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert g.gemm_f32_release() == 0
    graphs = []
    for s, w in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = _step(g, s, w)
        graphs.append((graph, out))
    big = _args(b, 4000, kind, 9, 2056)
    with torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        _step(g, *big)
    torch.cuda.synchronize()
    assert g.gemm_f32_release() == 0
    for seed in (1, 2):
        for (s, w), r in zip(args, sizes):
            _refill(s, w, *_args(b, r, kind, r + 1000 * seed))
        want = [_step(g, s, w) for s, w in args]
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
            with torch.cuda.stream(st):
                _step(g, *big)
        torch.cuda.synchronize()
        for (_, out), expected in zip(graphs, want):
            assert all(torch.equal(x, y) for x, y in zip(out, expected))
    assert g.gemm_f32_status(None) == (0, 0)


def test_two_graphs_of_one_stream_at_once():
    """Their scratch is their own: replayed on two streams at the same time."""
    import torch
    from tests import _block as b
    g = lib()
    args = [_args(b, 3000, "bf16", i) for i in range(2)]
    want = [_step(g, *a) for a in args]
    st, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for a in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = _step(g, *a)
        graphs.append((graph, out))
    for _ in range(20):
        for (graph, _), other in zip(graphs, others):
            with torch.cuda.stream(other):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), expected in zip(graphs, want):
        assert all(torch.equal(x, y) for x, y in zip(out, expected))


@pytest.mark.parametrize("shared", [True, False])
def test_threads(shared):
    """Host threads with calls of different sizes, on one stream or on one each."""
    import torch
    from tests import _block as b
    g = lib()
    args = [_args(b, 300 + 700 * i, "bf16", i) for i in range(4)]
    want = [_step(g, *a) for a in args]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    wrong = []

    def work(i):
        st = one if shared else torch.cuda.Stream()
        for _ in range(10):
            with torch.cuda.stream(st):
                out = _step(g, *args[i])
                same = torch.stack([(x == y).all() for x, y in zip(out, want[i])])
            st.synchronize()
            if not bool(same.all()):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and g.gemm_f32_status(None) == (0, 0)


def test_given_streams():
    """Calls queued on a stream that is not the current one."""
    import torch
    from tests import _block as b
    g = lib()
    s, w = _args(b, 700, "f32", 3)
    want = _step(g, s, w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y, h, stats = g.block_norm(s["branch"], s["residual"], s["weight"], s["bias"], stream=st, **s["how"])
    kept_y, kept_h, kept_b = (g.checkpoint(t, stream=st) for t in (y, h, s["branch"]))
    dw = g.weight_grad(w, kept_y, stream=st.cuda_stream)
    grads = g.block_norm_grad(s["dy"], s["dh"], kept_h, kept_b, stats, s["weight"], stream=st, **s["how"])
    back = g.restore(kept_h, stream=st)
    st.synchronize()
    got = [y, h, stats, kept_y.codes.view(torch.uint8), kept_y.exponents[:, :1], back, dw] + [v for v in grads if v is not None]
    assert all(torch.equal(x, v) for x, v in zip(got, want))


def test_in_an_autograd_function():
    """A custom autograd function of these calls against automatic differentiation in 64 bits: each result is within a few
    units of fp32 of its terms, of which 1e-5 of a gradient's size is allowed."""
    import torch
    from tests import _block as b
    g = lib()
    s = b.inputs(200, 520, "f32", "f32", "rms", "channel", True, 4)
    how = s["how"]
    names = ("branch", "residual", "weight", "post_weight", "gate")
    leaves = [s["branch"], s["residual"], s["weight"], how["post_weight"], how["gate"]]
    leaves = [t.clone().requires_grad_() for t in leaves]

    class End(torch.autograd.Function):
        @staticmethod
        def forward(ctx, branch, residual, weight, post_weight, gate):
            y, h, stats = g.block_norm(branch, residual, weight, kind="rms", post=True, post_weight=post_weight, gate=gate)
            ctx.save_for_backward(branch, h, stats, weight, post_weight, gate)
            return y, h

        @staticmethod
        def backward(ctx, dy, dh):
            branch, h, stats, weight, post_weight, gate = ctx.saved_tensors
            d = g.block_norm_grad(dy.contiguous(), dh.contiguous(), h, branch, stats, weight, kind="rms", post=True,
                                  post_weight=post_weight, gate=gate)
            return d.dbranch, d.dresidual, d.dweight, d.dpost_weight, d.dgate

    def step():
        y, h = End.apply(*leaves)
        return torch.autograd.grad((y * s["dy"]).sum() + (h * s["dh"]).sum(), leaves)

    got = step()
    d = [t.detach().double().requires_grad_() for t in leaves]
    rms = lambda t: t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-5)  # noqa: E731
    h = d[1] + d[4] * rms(d[0]) * d[3]
    y = rms(h) * d[2]
    exact = torch.autograd.grad((y * s["dy"].double()).sum() + (h * s["dh"].double()).sum(), d)
    for name, x, v in zip(names, got, exact):
        assert float((x.double() - v).norm()) <= 1e-5 * float(v.norm()), name


@pytest.mark.parametrize("rows", [9, 600])
def test_a_scratch_that_holds_anything(rows):
    """Memory that an allocation returns is not zero: every word of the scratch holds 3.0 before the call."""
    import torch
    from tests import _block as b
    from tests.test_gpu_lm_scratch import _scratch
    g = lib()
    s, w = _args(b, rows, "bf16", rows)
    one, threes = torch.ones((1, 1), device="cuda"), torch.full((1, 1 << 22), 3.0, device="cuda")
    want = _step(g, s, w)
    at = _scratch(0, 1 << 24)
    g.check(g.gemm_f32(one, threes, at, 1, 1 << 22, 1))
    assert all(torch.equal(x, v) for x, v in zip(_step(g, s, w), want))
