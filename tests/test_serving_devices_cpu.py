"""Decode-step calls and the device their tensors lie on: everything on one,
kernels launched with it as the current device. Shown without a GPU, with
tensors that claim to lie on one (of two)."""
import contextlib

import pytest

import bit_unstructured_sparse_amd as bsp
from test_serving_streams_cpu import (OnDevice, Stream, World, _adapters, _attend, _cache, _f16, _gather, _matrix,
                                      _tensor, _w4a4)

torch = pytest.importorskip("torch")


class OnAnother(OnDevice):
    device = torch.device("cuda:1")

    def get_device(self):
        return 1


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def _append(stream):
    bsp.kv_append(_cache(), _tensor((5, 2, 64), torch.float16), _tensor((5, 2, 64), torch.float16),
                  _tensor((5,), torch.int64), stream=stream)


CALLS = [_append, _gather, _attend, _f16, _w4a4]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_launched_with_the_tensors_device_as_the_current_one(call, current, world, monkeypatch):
    device = [current]

    @contextlib.contextmanager
    def switch(index):
        before, device[0] = device[0], index
        yield
        device[0] = before

    monkeypatch.setattr(torch.cuda, "device", switch)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: device[0], raising=False)
    seen = []
    get = type(world.lib).__getattr__

    def noting(self, name):
        fn = get(self, name)
        return fn if name.endswith("_bytes") else lambda *a: (seen.append(device[0]), fn(*a))[1]

    monkeypatch.setattr(type(world.lib), "__getattr__", noting)
    call(None)
    assert seen == [0] and device == [current]


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device(call, world):
    other = Stream(5)
    other.device_index = 1
    with pytest.raises(ValueError):
        call(other)
    assert not world.lib.calls


def test_a_workspace_on_another_device(world):
    ws = _tensor((1 << 20,), torch.uint8).as_subclass(OnAnother)
    i32 = torch.int32
    calls = [lambda: bsp.attention_tree(_tensor((1, 4, 64), torch.float16), _cache(), _tensor((1, 2), i32),
                                        _tensor((1,), i32), _tensor((2,), i32), 1, workspace=ws),
             lambda: bsp.spmm_f16_lora(_matrix(bsp.FP16, 64, 128), _tensor((8, 128), torch.float16),
                                       _adapters(64, 128), _tensor((8,), i32), workspace=ws),
             lambda: bsp.spmm_w4a4_dq_lora(_matrix(bsp.INT4, 64, 128), _tensor((8, 64), torch.uint8),
                                           _tensor((8, 128), torch.float16), _tensor((64,), torch.float32),
                                           _tensor((8,), torch.float32), _adapters(64, 128), _tensor((8,), i32),
                                           workspace=ws)]
    for call in calls:
        with pytest.raises(ValueError, match="workspace"):
            call()
    assert not world.lib.calls


@pytest.mark.parametrize("part", ["bitmaps", "offsets", "payload"])
def test_a_projection_on_another_device(part, world):
    W = _matrix(bsp.FP16, 64, 128)
    setattr(W, part, getattr(W, part).as_subclass(OnAnother))
    with pytest.raises(ValueError, match="projection"):
        bsp.spmm_f16_lora(W, _tensor((8, 128), torch.float16), _adapters(64, 128), _tensor((8,), torch.int32))
    W = _matrix(bsp.INT4, 64, 128)
    setattr(W, part, getattr(W, part).as_subclass(OnAnother))
    with pytest.raises(ValueError, match="projection"):
        bsp.spmm_w4a4_dq_lora(W, _tensor((8, 64), torch.uint8), _tensor((8, 128), torch.float16),
                              _tensor((64,), torch.float32), _tensor((8,), torch.float32), _adapters(64, 128),
                              _tensor((8,), torch.int32))
    assert not world.lib.calls
