"""What the decode-step calls allocate for themselves belongs to the stream
they run on. Shown without a GPU: tensors that claim to lie on one, a library
that launches nothing, and a record of the stream of each allocation."""
import contextlib

import pytest

import bit_unstructured_sparse_amd as bsp

torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda:0")

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.used_on = stream


def on_device(t):
    return t.as_subclass(OnDevice)


class Stream:
    device_index = 0

    def __init__(self, handle):
        self.cuda_stream = handle


class Library:
    """The size queries of the library; every other entry point notes its call."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return bsp.OK
        return call


class World:
    def __init__(self, monkeypatch):
        self.default, self.side = Stream(11), Stream(22)
        self.now, self.made = self.default, []
        self.lib = Library(bsp.load_library())
        monkeypatch.setattr(bsp, "load_library", lambda: self.lib)
        monkeypatch.setattr(torch.cuda, "stream", self.on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.now)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: self.now.cuda_stream, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
        for name in ("empty", "zeros", "empty_like"):
            monkeypatch.setattr(torch, name, self.maker(getattr(torch, name)))

    @contextlib.contextmanager
    def on(self, stream):
        before, self.now = self.now, stream
        yield
        self.now = before

    def maker(self, make):
        def made(*args, device=None, **kw):
            t = on_device(make(*args, **kw))
            self.made.append((t, self.now))
            return t
        return made


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def _tensor(shape, dtype):
    return on_device(torch.ones(shape, dtype=dtype))


def _adapters(M, K, R=16):
    return bsp.LoraAdapters(_tensor((2, R, K), torch.float16), _tensor((2, M, R), torch.float16))


def _matrix(dtype, M, K):
    return bsp.DeviceMatrix(dtype, M, K, M * K // 2, _tensor((M * ((K + 63) // 64),), torch.int64),
                            _tensor((M * ((K + 63) // 64) + 1,), torch.int32), _tensor((M * K,), torch.uint8))


def _f16(stream):
    return bsp.spmm_f16_lora(_matrix(bsp.FP16, 64, 11008), _tensor((8, 11008), torch.float16), _adapters(64, 11008),
                             _tensor((8,), torch.int32), stream=stream)


def _w4a4(stream):
    return bsp.spmm_w4a4_dq_lora(_matrix(bsp.INT4, 64, 128), _tensor((8, 64), torch.uint8),
                                 _tensor((8, 128), torch.float16), _tensor((64,), torch.float32),
                                 _tensor((8,), torch.float32), _adapters(64, 128), _tensor((8,), torch.int32),
                                 stream=stream)


def _cache():
    k = _tensor((2, 2, 16, 64), torch.uint8)
    w = _tensor((2, 2, 16), torch.int32)
    return bsp.KVCache(bsp.INT8, k, k.clone().as_subclass(OnDevice), w, w.clone().as_subclass(OnDevice))


def _gather(stream):
    return bsp.kv_gather(_cache(), _tensor((5,), torch.int64), stream=stream)


def _attend(stream):
    i32 = torch.int32
    return bsp.attention_tree(_tensor((1, 4, 64), torch.float16), _cache(), _tensor((1, 2), i32), _tensor((1,), i32),
                              _tensor((2,), i32), 1, stream=stream)


# (call, tensors it makes: outputs, then the workspace)
CALLS = [(_f16, 2), (_w4a4, 2), (_gather, 2), (_attend, 1)]


@pytest.mark.parametrize("call,count", CALLS, ids=lambda v: getattr(v, "__name__", None))
def test_made_on_the_stream_of_the_call(call, count, world):
    out = call(world.side)
    assert len(world.made) == count
    assert all(stream is world.side for _, stream in world.made)
    (_, args), = world.lib.calls
    assert args[-1] == world.side.cuda_stream
    # the caller reads the outputs on the stream it is on
    for t in out if isinstance(out, tuple) else (out,):
        assert t.used_on is world.default


@pytest.mark.parametrize("call,count", CALLS, ids=lambda v: getattr(v, "__name__", None))
def test_made_on_the_current_stream_without_one(call, count, world):
    with torch.cuda.stream(world.side):
        call(None)
    assert [stream for _, stream in world.made] == [world.side] * count
    (_, args), = world.lib.calls
    assert args[-1] == world.side.cuda_stream
