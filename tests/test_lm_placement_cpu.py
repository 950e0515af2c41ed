"""Where the calls on torch tensors run, on stand-ins for the tensors, the
devices and the library: on the tensors' device, whichever is current, and on
the stream that is given, which owns what is allocated; and what becomes of a
call for whose scratch there is no memory."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")


class Tensor:
    """The parts of a CUDA tensor that the checks look at."""

    def __init__(self, shape, dtype=torch.float32, dev=0):
        self.shape, self.dtype, self.dev = tuple(shape), dtype, dev
        self.is_cuda, self.device = True, "cuda:%d" % dev

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class Stream:
    def __init__(self, device_index, cuda_stream):
        self.device_index, self.cuda_stream = device_index, cuda_stream


@pytest.fixture
def world(monkeypatch):
    """The current device, each device's current stream, and what was called and allocated where."""
    import accelerator_row_major_gb300 as g
    from accelerator_row_major_gb300 import _binding, _lm
    state = types.SimpleNamespace(device=0, streams={0: Stream(0, 10), 1: Stream(1, 20)}, calls=[], made=[], answers=[], emptied=0, capturing=False)

    def empty(shape, dtype=None, device=None, **_):
        dev = int(str(device)[-1])
        state.made.append((dev, state.streams[dev].cuda_stream))
        return Tensor(shape if isinstance(shape, tuple) else (shape,), dtype, dev)

    def entry(name):
        def call(*args):
            state.calls.append((name, state.device, state.streams[state.device].cuda_stream, args))
            return state.answers.pop(0) if state.answers else 0
        return call

    @contextlib.contextmanager
    def device(d):
        state.device, before = d, state.device
        yield
        state.device = before

    @contextlib.contextmanager
    def stream(s):
        before, had = state.device, state.streams[s.device_index]
        state.device, state.streams[s.device_index] = s.device_index, s
        yield
        state.device, state.streams[s.device_index] = before, had

    class Library:
        def __getattr__(self, name):
            return entry(name)

    def empty_cache():
        state.emptied += 1

    monkeypatch.setattr(torch.cuda, "empty_cache", empty_cache)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t, **_: empty(t.shape, t.dtype, t.device))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream(device, handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d: Stream(d, 0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: state.streams[int(str(d)[-1])])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.device, raising=False)
    monkeypatch.setattr(_lm, "_current_device", lambda: state.device)
    monkeypatch.setattr(_lm, "_raw_stream", lambda d: state.streams[d].cuda_stream)
    monkeypatch.setattr(_binding, "lib", lambda: Library())
    monkeypatch.setattr(_lm, "lib", lambda: Library())
    state.g = g
    return state


def _calls(g, dev):
    x, w, y = Tensor((4, 8), dev=dev), Tensor((16, 8), dev=dev), Tensor((4,), torch.int64, dev)
    weight, stat, square = Tensor((8,), dev=dev), Tensor((4,), dev=dev), Tensor((8, 8), dev=dev)
    return {"gemm_f32_layer_norm": lambda **k: g.layer_norm(x, weight, weight, **k),
            "gemm_f32_layer_norm_grad": lambda **k: g.layer_norm_grad(x, x, weight, stat, stat, **k),
            "gemm_f32_vocab_loss": lambda **k: g.vocab_loss(x, w, y, **k),
            "gemm_f32_vocab_loss_grad": lambda **k: g.vocab_loss_grad(x, w, y, **k),
            "gemm_f32_ex": lambda **k: g.matmul(x, square, **k)}


NAMES = sorted(_calls(None, 0))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, 1])
def test_a_call_runs_on_its_tensors_device(world, name, current):
    world.device = current
    _calls(world.g, 1)[name]()
    (called, device, stream, args), = world.calls
    assert (called, device, stream, args[-1]) == (name, 1, 20, 20)
    assert set(world.made) == {(1, 20)} and world.device == current


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("given,handle", [(lambda d: Stream(d, 77), 77), (lambda d: 78, 78), (lambda d: 0, 0)])
def test_what_a_call_allocates_belongs_to_its_stream(world, name, dev, given, handle):
    _calls(world.g, dev)[name](stream=given(dev))
    (called, device, stream, args), = world.calls
    assert (called, device, stream, args[-1]) == (name, dev, handle, handle)
    assert set(world.made) == {(dev, handle)}
    assert world.device == 0 and world.streams[dev].cuda_stream == 10 * (dev + 1)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(world, name):
    with pytest.raises(ValueError):
        _calls(world.g, 1)[name](stream=Stream(0, 77))
    assert not world.calls


@pytest.mark.parametrize("name", ["gemm_f32_layer_norm_grad", "gemm_f32_vocab_loss", "gemm_f32_vocab_loss_grad"])
@pytest.mark.parametrize("capturing,answers,calls", [(False, [-5], 2), (False, [-5, -5], 2), (True, [-5], 1), (False, [-3], 1)])
def test_memory_that_torch_holds_is_asked_for_once(world, name, capturing, answers, calls):
    world.answers, world.capturing = list(answers), capturing
    if len(answers) == calls:
        with pytest.raises(world.g.GemmError) as e:
            _calls(world.g, 0)[name]()
        assert e.value.code == answers[0]
    else:
        _calls(world.g, 0)[name]()
    assert len(world.calls) == calls and world.emptied == calls - 1
