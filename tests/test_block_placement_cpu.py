"""Where the calls of _block run, on the stand-ins of
tests/test_lm_placement_cpu.py: on the tensors' device, whichever is current,
on the stream that is given, which owns what is allocated; what they refuse;
and what becomes of a call for whose scratch there is no memory."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_lm_placement_cpu import Stream, Tensor, world  # noqa: E402,F401

F8, U8, BF16 = torch.float8_e4m3fn, torch.uint8, torch.bfloat16


def _kept(g, rows=4, width=40, dtype=torch.float32, dev=0, **kw):
    codes, exponents = kw.get("codes", (rows, 64)), kw.get("exponents", (rows, 16))
    return g.Checkpoint(Tensor(codes, kw.get("ctype", F8), dev), Tensor(exponents, kw.get("etype", U8), kw.get("edev", dev)), width, dtype)


def _calls(g, dev):
    x, dy, w, stats = Tensor((4, 40), dev=dev), Tensor((4, 24), dev=dev), Tensor((40,), dev=dev), Tensor((4, 4), dev=dev)
    how = dict(post=True, post_weight=w, post_bias=w, gate=w)
    return {"gemm_f32_block_norm": lambda **k: g.block_norm(x, x, w, w, **how, **k),
            "gemm_f32_block_norm_grad": lambda **k: g.block_norm_grad(x, x, x, _kept(g, dev=dev), stats, w, **how, **k),
            "gemm_f32_checkpoint": lambda **k: g.checkpoint(x, **k),
            "gemm_f32_restore": lambda **k: g.restore(_kept(g, dev=dev), **k),
            "gemm_f32_weight_grad": lambda **k: g.weight_grad(dy, _kept(g, dev=dev), **k)}


class _Names:
    def __getattr__(self, name):
        return lambda *a, **k: None


NAMES = sorted(_calls(_Names(), 0))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, 1])
def test_a_call_runs_on_its_tensors_device(world, name, current):  # noqa: F811
    world.device = current
    _calls(world.g, 1)[name]()
    (called, device, stream, args), = world.calls
    assert (called, device, stream, args[-1]) == (name, 1, 20, 20)
    assert set(world.made) == {(1, 20)} and world.device == current


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("given,handle", [(lambda d: Stream(d, 77), 77), (lambda d: 78, 78), (lambda d: 0, 0)])
def test_what_a_call_allocates_belongs_to_its_stream(world, name, dev, given, handle):  # noqa: F811
    _calls(world.g, dev)[name](stream=given(dev))
    (called, device, stream, args), = world.calls
    assert (called, device, stream, args[-1]) == (name, dev, handle, handle)
    assert set(world.made) == {(dev, handle)}
    assert world.device == 0 and world.streams[dev].cuda_stream == 10 * (dev + 1)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(world, name):  # noqa: F811
    with pytest.raises(ValueError):
        _calls(world.g, 1)[name](stream=Stream(0, 77))
    assert not world.calls


@pytest.mark.parametrize("name", ["gemm_f32_block_norm_grad", "gemm_f32_weight_grad"])
@pytest.mark.parametrize("capturing,answers,calls", [(False, [-5], 2), (False, [-5, -5], 2), (True, [-5], 1), (False, [-3], 1)])
def test_memory_that_torch_holds_is_asked_for_once(world, name, capturing, answers, calls):  # noqa: F811
    world.answers, world.capturing = list(answers), capturing
    if len(answers) == calls:
        with pytest.raises(world.g.GemmError) as e:
            _calls(world.g, 0)[name]()
        assert e.value.code == answers[0]
    else:
        _calls(world.g, 0)[name]()
    assert len(world.calls) == calls and world.emptied == calls - 1


def test_what_the_calls_refuse(world):  # noqa: F811
    g = world.g
    x, b, w, s = Tensor((4, 40)), Tensor((4, 40), BF16), Tensor((40,)), Tensor((2, 4))
    wb, dy = Tensor((40,), BF16), Tensor((4, 24))
    bad = [lambda: g.block_norm(x, b), lambda: g.block_norm(x, Tensor((4, 41))), lambda: g.block_norm(x, Tensor((4, 40), dev=1)),
           lambda: g.block_norm(x, x, w, Tensor((41,))), lambda: g.block_norm(x, x, wb), lambda: g.block_norm(b, b, w, wb),
           lambda: g.block_norm(x, x, kind="batch"), lambda: g.block_norm(x, x, post_weight=w), lambda: g.block_norm(x, x, post_bias=w),
           lambda: g.block_norm(x, x, w, w, kind="rms"), lambda: g.block_norm(x, x, kind="rms", post=True, post_bias=w),
           lambda: g.block_norm(x, x, gate=b), lambda: g.block_norm(x, x, gate=Tensor((4, 1))), lambda: g.block_norm(x, x, gate=Tensor((4,))),
           lambda: g.block_norm(b, b, w, gate=wb), lambda: g.block_norm(x, x, out=b), lambda: g.block_norm(x, x, out_h=Tensor((4, 39))),
           lambda: g.block_norm_grad(x, b, x, None, s), lambda: g.block_norm_grad(x, x, b, None, s),
           lambda: g.block_norm_grad(x, x, x, None, s, gate=w), lambda: g.block_norm_grad(x, x, x, None, s, post=True),
           lambda: g.block_norm_grad(x, x, x, x, s, post=True), lambda: g.block_norm_grad(x, x, x, None, Tensor((4, 4))),
           lambda: g.block_norm_grad(x, x, x, None, Tensor((2, 4), BF16)), lambda: g.block_norm_grad(x, x, x, None, Tensor((2, 4), dev=1)),
           lambda: g.block_norm_grad(x, x, _kept(g, dtype=BF16), None, s), lambda: g.block_norm_grad(x, x, _kept(g, width=39), None, s),
           lambda: g.block_norm_grad(x, x, _kept(g, rows=5), None, s), lambda: g.block_norm_grad(x, x, _kept(g, dev=1), None, s),
           lambda: g.restore(_kept(g, codes=(4, 40))), lambda: g.restore(_kept(g, exponents=(4, 2))), lambda: g.restore(_kept(g, ctype=U8)),
           lambda: g.restore(_kept(g, etype=torch.int8)), lambda: g.restore(_kept(g, edev=1)), lambda: g.restore(_kept(g, width=0)),
           lambda: g.restore(_kept(g, dtype=torch.float16)), lambda: g.restore(_kept(g), out=b), lambda: g.restore(_kept(g), out=Tensor((4, 41))),
           lambda: g.weight_grad(dy, _kept(g, rows=5)), lambda: g.weight_grad(dy, _kept(g, dtype=BF16)), lambda: g.weight_grad(dy, _kept(g, dev=1)),
           lambda: g.weight_grad(dy, _kept(g), accumulate=True), lambda: g.weight_grad(dy, _kept(g), out=Tensor((24, 41))),
           lambda: g.weight_grad(dy, _kept(g), out=Tensor((24, 40), BF16)),
           lambda: g.weight_grad(Tensor((4, 24), BF16), _kept(g, dtype=BF16), out=Tensor((24, 40), BF16), accumulate=True),
           lambda: g.weight_grad(dy, _kept(g), out=Tensor((24, 40), dev=1))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert not world.calls


def test_what_reaches_the_library(world):  # noqa: F811
    """A gradient's optional outputs: what the block does not have is a null pointer, and one tensor serves for two."""
    g = world.g
    x, w, s = Tensor((4, 40)), Tensor((40,)), Tensor((2, 4))
    d = g.block_norm_grad(x, None, x, None, s, w, kind="rms")
    args = world.calls.pop()[3]
    assert d.dbranch is d.dresidual and (d.dbias, d.dgate, d.dpost_weight, d.dpost_bias) == (None,) * 4
    assert args[3] == 0 and args[6] is None and args[8] == 0 and args[12] == 0 and args[15:18] == (0, 0, 0)
    d = g.block_norm_grad(x, x, x, x, s, w, gate=x, branch_scale=0.5)
    args = world.calls.pop()[3]
    assert d.dbranch is not d.dresidual and d.dgate.shape == (4, 40) and d.dbias.shape == (40,)
    assert args[6] is not None and args[8] and args[12] and args[15]
