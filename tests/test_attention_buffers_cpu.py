"""Where the binding of the attention calls makes its buffers and what it asks of the library, with stand-ins for
tensors, streams, devices and the library (no GPU)."""

import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
vq3 = pytest.importorskip("bit_vector_lut_gb300.vq3", reason="libvq3.so not built")

DEVICE = 1  # of the tensors; device 0 is the current one unless a test says otherwise
BYTES = {0: 1 << 20, 1: 3 << 20}  # workspace that a call needs on either device


class Tensor:
    def __init__(self, shape, dtype, strides=None, device=DEVICE, contiguous=True):
        self.shape, self.dtype, self.index, self.contiguous = torch.Size(shape), dtype, device, contiguous
        self.strides = strides or torch.empty(shape, device="meta").stride()
        self.device = f"cuda:{device}"
        self.recorded = []

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.strides

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def is_contiguous(self):
        return self.contiguous

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x10000

    def record_stream(self, s):
        self.recorded.append(s)


class Stream:
    def __init__(self, name, device=DEVICE, handle=77):
        self.name, self.device_index, self.cuda_stream = name, device, handle


class World:
    """The current device and stream, the buffers made and the library's calls, in order."""

    def __init__(self, monkeypatch):
        self.device, self.main = 0, Stream("main", handle=5)
        self.stream, self.made, self.calls = self.main, [], []
        self.answers = []  # statuses of the next calls, 0 when they run out

        @contextlib.contextmanager
        def on_stream(s):
            was = self.stream, self.device
            self.stream, self.device = s, s.device_index
            yield
            self.stream, self.device = was

        @contextlib.contextmanager
        def on_device(i):
            was, self.device = self.device, i
            yield
            self.device = was

        def empty(*shape, dtype, device):
            t = Tensor(shape[0] if isinstance(shape[0], (tuple, torch.Size)) else shape, dtype)
            self.made.append((t, self.stream))
            return t

        def call(name):
            def f(*args):
                self.calls.append((name, self.device, self.stream, args))
                return self.answers.pop(0) if self.answers else 0
            return f

        monkeypatch.setattr(torch.cuda, "stream", on_stream)
        monkeypatch.setattr(torch.cuda, "device", on_device)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: self.stream)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.device, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: self.stream.cuda_stream, raising=False)
        monkeypatch.setattr(vq3, "_empty", empty)
        monkeypatch.setattr(vq3, "lib", types.SimpleNamespace(
            vq3_paged_plan=call("plan"), vq3_paged_attention=call("paged"), vq3_prompt_attention=call("prompt"),
            vq3_kv_append=call("append"), vq3_last_error=lambda: b"refused",
            vq3_attention_workspace_bytes=lambda *a: BYTES[self.device]))


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def ints(*shape):
    return Tensor(shape, torch.int32)


def half(*shape):
    return Tensor(shape, torch.float16)


def run_plan(**kw):
    return tuple(vq3.paged_plan(ints(3), ints(3), ints(3, 5), ints(9), ints(2), 16, 20, **kw))


def run_paged(**kw):
    return (vq3.paged_attention(half(7, 8, 128), half(9, 16, 2, 128), half(9, 16, 2, 128), ints(3, 5), ints(4), ints(3),
                                max_new=4, **kw),)


def run_prompt(**kw):
    return (vq3.prompt_attention(half(7, 8, 128), half(7, 2, 128), half(7, 2, 128), ints(4), max_new=4, **kw),)


CALLS = [run_plan, run_paged, run_prompt]


@pytest.mark.parametrize("run", CALLS)
def test_buffers_come_from_the_stream_that_writes_them(world, run):
    side = Stream("side")
    got = run(stream=side)
    assert world.made and all(s is side for _, s in world.made)
    assert world.calls[-1][3][-1] == side.cuda_stream
    # what is handed back is used on the current stream: not given out again before that
    assert all(t.recorded == [world.main] for t in got)
    assert world.stream is world.main and world.device == 0


@pytest.mark.parametrize("run", CALLS)
def test_without_a_stream_the_current_one_is_used(world, run):
    got = run()
    assert world.made and all(s is world.main for _, s in world.made)
    assert world.calls[-1][3][-1] == 5 and not any(t.recorded for t in got)


@pytest.mark.parametrize("run", CALLS)
def test_the_current_stream_given_by_name(world, run):
    got = run(stream=world.main)
    assert all(s is world.main for _, s in world.made) and not any(t.recorded for t in got)


@pytest.mark.parametrize("run", [run_paged, run_prompt])
@pytest.mark.parametrize("current", [0, 1])
def test_workspace_is_sized_on_the_tensors_device(world, run, current):
    # the devices need not have the same number of SMs, on which the size depends
    world.device = current
    run()
    name, device, _, args = world.calls[-1]
    assert device == DEVICE and args[-2] == BYTES[DEVICE] and world.device == current


@pytest.mark.parametrize("run", [run_paged, run_prompt])
def test_buffers_of_the_callers_on_a_stream_of_the_callers(world, run):
    # nothing is made: only the call goes to that stream and device
    side, out, ws = Stream("side"), half(7, 8, 128), Tensor((1 << 22,), torch.uint8)
    assert run(out=out, ws=ws, stream=side)[0] is out and not world.made and not out.recorded
    name, device, stream, args = world.calls[-1]
    assert device == DEVICE and args[-1] == side.cuda_stream and world.stream is world.main
    world.device = DEVICE
    run(out=out, ws=ws, stream=side)
    assert world.calls[-1][2] is world.main and world.calls[-1][3][-1] == side.cuda_stream
    run(out=out, stream=side)  # a workspace is made
    assert [s for _, s in world.made] == [side] and not out.recorded
    with pytest.raises(vq3.Vq3Error, match="stream of CUDA device 0"):
        run(out=out, ws=ws, stream=Stream("other", device=0))


def test_every_call_runs_on_the_tensors_device(world):
    run_plan()
    vq3.kv_append(half(7, 2, 128), half(7, 2, 128), Tensor((7,), torch.int64), half(9, 16, 2, 128), half(9, 16, 2, 128))
    assert [(c[0], c[1]) for c in world.calls] == [("plan", DEVICE), ("append", DEVICE)] and world.device == 0


@pytest.mark.parametrize("run", CALLS)
def test_a_stream_of_another_device_is_refused(world, run):
    with pytest.raises(vq3.Vq3Error, match="stream of CUDA device 0"):
        run(stream=Stream("other", device=0))
    assert not world.calls and not world.made


@pytest.mark.parametrize("run", [run_paged, run_prompt])
def test_a_workspace_that_the_call_cannot_write_is_refused(world, run):
    for ws in (Tensor((1 << 22,), torch.uint8, device=0),      # another device's
               Tensor((1 << 22,), torch.uint8, device=-1),     # host memory
               Tensor((1 << 22,), torch.uint8, strides=(0,), contiguous=False)):  # one byte, expanded
        with pytest.raises(vq3.Vq3Error, match="ws must be"):
            run(ws=ws)
    assert not world.calls
    # its size in bytes, whatever its type
    run(ws=Tensor((1 << 20,), torch.float32))
    assert world.calls[-1][3][-2] == 4 << 20
