"""What the classes of the low-bit linear layer hand to the library: which memory a call reads and writes. The library's
calls are recorded here, not made."""
import ctypes

import numpy as np
import pytest
import torch

from bit_quantization_block_amd import lq


class Recorder:
    """The library's own sizes; the calls that would launch only leave their arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        real = getattr(lq.load(), name)
        if name.endswith("_bytes"):
            return real

        def call(desc, *args):
            self.calls.append((name, desc._obj, *[a.value if isinstance(a, ctypes.c_void_p) else a for a in args]))
            return 0

        return call


class OnGpu(torch.Tensor):
    """A host tensor that says it is the GPU's."""
    is_cuda = True


def device_tensor(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture(autouse=True)
def stream(monkeypatch):
    monkeypatch.setattr(lq, "_stream_of", lambda device, stream: 0)
    monkeypatch.setattr(lq, "_stream", lambda stream: 0)


@pytest.fixture
def layer():
    lib = Recorder()
    made = lq.Mx4Linear(device_tensor(64, 64), rows=8, lib=lib)
    lib.calls.clear()
    return made


def spans(t):
    size = t.element_size()
    return {t.data_ptr() + (i * t.stride(0) + j) * size + b for i in range(t.shape[0]) for j in range(t.shape[1]) for b in range(size)}


def test_shared_memory_is_seen_byte_by_byte():
    rng = np.random.default_rng(1)
    flat = torch.zeros(400, dtype=torch.uint8)
    met = 0
    for _ in range(4000):
        pair = []
        for _ in range(2):
            dtype = [torch.uint8, torch.float16, torch.float32][rng.integers(3)]
            size = dtype.itemsize
            rows, cols = rng.integers(0, 5), rng.integers(0, 6)
            ld = cols + rng.integers(0, 9)
            start = rng.integers(0, 40) * size
            pair.append(flat[start:start + (400 - start) // size * size].view(dtype).as_strided((rows, cols), (ld, 1)))
        a, b = pair
        want = bool(spans(a) & spans(b))
        met += want
        assert lq._share(a, b) == want and lq._share(b, a) == want, (a.shape, a.stride(), b.shape, b.stride())
    assert 500 < met < 3500


def args_of(layer, name):
    return [c for c in layer.lib.calls if c[0] == name][-1]


@pytest.mark.parametrize("kind,name,reads,writes", [("forward", "lq_mx4_linear", 2, 5), ("dgrad", "lq_mx4_dgrad", 2, 5)])
def test_a_result_can_be_the_next_calls_input(layer, kind, name, reads, writes):
    """The layer's buffer, handed out as a result, is not overwritten by the call that reads it."""
    call = getattr(layer, kind)
    for rows in (8, 3):
        y = call(device_tensor(8, 64))[:rows].as_subclass(OnGpu)
        for _ in range(4):
            z = call(y)
            c = args_of(layer, name)
            assert c[reads] == y.data_ptr() and c[writes] == z.data_ptr()
            assert not lq._share(y, z) and z.shape == (rows, 64)
            y = z.as_subclass(OnGpu)
    assert len(layer._buffers) == 2


@pytest.mark.parametrize("kind", ["forward", "dgrad"])
def test_out_may_not_be_the_input(layer, kind):
    call = getattr(layer, kind)
    x = device_tensor(8, 64)
    with pytest.raises(ValueError, match="share memory"):
        call(x, out=x)
    long = device_tensor(9, 64)
    with pytest.raises(ValueError, match="share memory"):
        call(long[:8], out=long[1:])
    assert not layer.lib.calls
    both = device_tensor(8, 136)                     # side by side: nothing shared
    call(both[:, :64], out=both[:, 72:])
    assert len(layer.lib.calls) == 1


def test_dw_in_is_the_result_or_apart_from_it(layer):
    kept = lq.Ckpt8.__new__(lq.Ckpt8)
    kept.rows, kept.cols, kept.fmt = 8, 64, "int8"
    kept.codes = kept.scales = device_tensor(8 * 64, dtype=torch.uint8)
    dy = device_tensor(8, 64)
    big = device_tensor(65, 64, dtype=torch.float32)
    layer.wgrad(dy, kept, dw_in=big[:64], out=big[:64])
    layer.wgrad(dy, kept, dw_in=layer.wgrad(dy, kept).as_subclass(OnGpu))
    assert len(layer.lib.calls) == 3
    with pytest.raises(ValueError, match="share memory"):
        layer.wgrad(dy, kept, dw_in=big[:64], out=big[1:])
    with pytest.raises(ValueError, match="share memory"):
        layer.wgrad(big.view(torch.bfloat16)[:8, :64], kept, out=big[:64])
    assert len(layer.lib.calls) == 3


def unit(rows, cols):
    act = lq.SwigluCkpt8.__new__(lq.SwigluCkpt8)
    act.torch, act.lib, act.rows, act.cols, act.dtype, act.fmt = torch, Recorder(), rows, cols, "bf16", "int8"
    act._t, act._kept, act.device, act._index = torch.bfloat16, (16, 16, 16, 16), torch.device("cpu"), None
    act._plans, act._buffers = {}, {}
    return act


def test_the_gated_unit_in_place_or_apart():
    act = unit(8, 64)
    big = device_tensor(9, 64)
    g, u = big[:8], device_tensor(8, 64)
    act.forward(g, u, out=g)
    act.forward(u, g, out=g)
    act.forward(act.forward(g, u).as_subclass(OnGpu), u)
    act.backward(g, out=(g, u))
    act.backward(u, out=(g, u))
    assert len(act.lib.calls) == 6
    for refused in (lambda: act.forward(g, u, out=big[1:]), lambda: act.forward(u, g, out=big[1:]),
                    lambda: act.backward(g, out=(big[1:], u)), lambda: act.backward(g, out=(u, big[1:])),
                    lambda: act.backward(u, out=(g, g)), lambda: act.backward(u, out=(g, big[1:]))):
        with pytest.raises(ValueError, match="share memory"):
            refused()
    assert len(act.lib.calls) == 6


def elsewhere(*shape, dtype=torch.bfloat16):
    """A tensor that says it is a GPU's, but another's."""
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnGpu)


def test_every_tensor_of_a_call_is_on_the_objects_device(layer):
    for device in ("cpu", torch.device("cpu"), "meta"):
        with pytest.raises(ValueError, match="GPU"):
            lq.Ckpt8(8, 64, device=device)
        with pytest.raises(ValueError, match="GPU"):
            lq.SwigluCkpt8(8, 64, device=device)
    kept = lq.Ckpt8.__new__(lq.Ckpt8)
    kept.rows, kept.cols, kept.fmt, kept.lib, kept._index = 8, 64, "int8", layer.lib, None
    kept.codes = kept.scales = elsewhere(8 * 64, dtype=torch.uint8)
    x, dy = device_tensor(8, 64), device_tensor(8, 64)
    for refused in (lambda: layer.forward(x, ckpt=kept), lambda: layer.wgrad(dy, kept), lambda: kept.save(x),
                    lambda: layer.load(elsewhere(64, 64)), lambda: layer.forward(elsewhere(7, 64)),
                    lambda: layer.forward(x, out=elsewhere(8, 64)), lambda: layer.dgrad(elsewhere(7, 64))):
        with pytest.raises(ValueError, match=" on "):
            refused()
    kept.codes = kept.scales = torch.empty(8 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="dw_in is on"):
        layer.wgrad(dy, kept, dw_in=elsewhere(64, 64, dtype=torch.float32))
    assert not layer.lib.calls


def test_calls_are_made_on_the_memorys_device(monkeypatch):
    """With several GPUs, one that is not the current device becomes it for the call."""
    now, seen = [0], []

    class At:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, now[0] = now[0], self.device

        def __exit__(self, *exc):
            now[0] = self.before

    class Lib:
        def lq_mx4_linear(self, *args):
            seen.append((now[0], args))
            return -3

    monkeypatch.setattr(torch.cuda, "device", At)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    for device in (0, 1, 1):
        assert lq._library(Lib(), device).lq_mx4_linear(5, 6) == -3
    assert seen == [(0, (5, 6)), (1, (5, 6)), (1, (5, 6))] and now == [0]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    lib = Lib()
    assert lq._library(lib, 0) is lib


def test_weights_and_checkpoints_go_on_their_devices_stream(layer, monkeypatch):
    monkeypatch.setattr(lq, "_stream_of", lambda device, stream: ("of", device, stream))
    layer.load(device_tensor(64, 64))
    kept = lq.Ckpt8.__new__(lq.Ckpt8)
    kept.rows, kept.cols, kept.fmt, kept.lib, kept._index = 8, 64, "int8", layer.lib, 3
    kept.codes = kept.scales = device_tensor(8 * 64, dtype=torch.uint8)
    kept.save(device_tensor(8, 64))
    kept.save(device_tensor(8, 64), stream=77)
    assert [c[-1] for c in layer.lib.calls] == [("of", None, None), ("of", 3, None), ("of", 3, 77)]


def test_memory_comes_from_the_calls_streams_pool(layer, monkeypatch):
    """Buffers and workspaces of a call on a stream of its own are not taken from the current stream's pool."""
    now, taken, empty = [5], [], torch.empty

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    class At:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, now[0] = now[0], self.s.cuda_stream

        def __exit__(self, *exc):
            now[0] = self.before

    def took(*args, **kw):
        taken.append(now[0])
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[0]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", At)
    monkeypatch.setattr(torch, "empty", took)
    x = device_tensor(8, 64)
    y = layer.forward(x, stream=9).as_subclass(OnGpu)
    layer.forward(y, stream=9)
    assert set(taken) == {9} and len(taken) == 3                    # result, workspace, the second buffer
    taken.clear()
    layer.dgrad(device_tensor(8, 64), stream=0)
    assert set(taken) == {0} and now == [5]
    taken.clear()
    act = unit(8, 64)
    act.forward(x, y, stream=9)
    assert taken == [9]
    act.backward(x, stream=5)
    act.backward(device_tensor(8, 64)[:, :64])
    assert taken == [9, 5, 5]


def test_inputs_that_wait_for_a_gradient_are_refused(layer):
    x = torch.zeros(8, 64, dtype=torch.bfloat16, requires_grad=True).as_subclass(OnGpu)
    plain = device_tensor(8, 64)
    act = unit(8, 64)
    kept = lq.Ckpt8.__new__(lq.Ckpt8)
    kept.rows, kept.cols, kept.fmt, kept.lib, kept._index = 8, 64, "int8", layer.lib, None
    kept.codes = kept.scales = torch.empty(8 * 64, dtype=torch.uint8)
    calls = [lambda: layer.forward(x), lambda: layer.dgrad(x), lambda: layer.wgrad(x, kept), lambda: kept.save(x),
             lambda: act.forward(x, plain), lambda: act.forward(plain, x), lambda: act.backward(x)]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    assert not layer.lib.calls and not act.lib.calls
    with torch.no_grad():
        for call in calls:
            call()
    layer.load(torch.nn.Parameter(torch.zeros(64, 64)).as_subclass(OnGpu))
    assert len(layer.lib.calls) == 5 and len(act.lib.calls) == 3
