"""The calls from the hidden states to the cache: what they allocate belongs to their stream, and they are
launched with their tensors' device as the current one. Shown without a GPU."""
import pytest

import bit_unstructured_sparse_amd as bsp
from test_serving_devices_cpu import OnAnother, test_launched_with_the_tensors_device_as_the_current_one as launched_on
from test_serving_streams_cpu import Stream, World, _cache, _tensor

torch = pytest.importorskip("torch")
I32, F16 = torch.int32, torch.float16


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def _pages(stream):
    pages = bsp.KVPages(_tensor((3, 4), I32), _tensor((3,), I32), _tensor((3,), I32), _tensor((10,), I32), 16)
    return bsp.kv_step(pages, None, _tensor((3,), I32), 8, stream=stream)


def _heads(stream):
    return bsp.qk_norm_rope(_tensor((5, 4, 64), F16), _tensor((5, 2, 64), F16), _tensor((5,), I32),
                            _tensor((32,), torch.int64), stream=stream)


def _append(stream):
    return bsp.qk_norm_rope_append(_tensor((5, 4, 64), F16), _tensor((5, 2, 64), F16), _tensor((5, 2, 64), F16),
                                   _tensor((5,), I32), _tensor((32,), torch.int64), _cache(),
                                   _tensor((5,), torch.int64), stream=stream)


def _quantise(stream):
    t = _tensor((5, 100), F16)
    return bsp.quantize_tokens(t, bsp.INT4, residual=_tensor((5, 100), F16), x16=True, stream=stream)


def _back(stream):
    return bsp.dequantize_tokens(_tensor((5, 50), torch.uint8), _tensor((5,), torch.float32), bsp.INT4, 100,
                                 stream=stream)


def _product(stream):
    W = bsp.DenseInt8(32, 64, _tensor((2048,), torch.uint8), _tensor((32,), torch.float32))
    return bsp.gemm_w8a8(W, _tensor((5, 64), torch.int8), _tensor((5,), torch.float32), stream=stream)


CALLS = [(_pages, 5), (_heads, 2), (_append, 1), (_quantise, 4), (_back, 1), (_product, 1)]
IDS = [c.__name__ for c, _ in CALLS]


@pytest.mark.parametrize("call,count", CALLS, ids=IDS)
def test_made_on_the_stream_of_the_call(call, count, world):
    out = call(world.side)
    assert len(world.made) == count and all(stream is world.side for _, stream in world.made)
    (_, args), = world.lib.calls
    assert args[-1] == world.side.cuda_stream
    for t in out if isinstance(out, tuple) else (out,):
        assert t.used_on is world.default


@pytest.mark.parametrize("call,count", CALLS, ids=IDS)
def test_made_on_the_current_stream_without_one(call, count, world):
    with torch.cuda.stream(world.side):
        call(None)
    assert [stream for _, stream in world.made] == [world.side] * count
    (_, args), = world.lib.calls
    assert args[-1] == world.side.cuda_stream


@pytest.mark.parametrize("call", [c for c, _ in CALLS], ids=IDS)
@pytest.mark.parametrize("current", [0, 1])
def test_launched_with_the_tensors_device(call, current, world, monkeypatch):
    launched_on(call, current, world, monkeypatch)


@pytest.mark.parametrize("call", [c for c, _ in CALLS], ids=IDS)
def test_a_stream_of_another_device(call, world):
    other = Stream(5)
    other.device_index = 1
    with pytest.raises(ValueError):
        call(other)
    assert not world.lib.calls


def test_tensors_of_another_device(world):
    far = lambda shape, dtype: _tensor(shape, dtype).as_subclass(OnAnother)
    pages = bsp.KVPages(_tensor((3, 4), I32), _tensor((3,), I32), _tensor((3,), I32), _tensor((10,), I32), 16)
    W = bsp.DenseInt8(32, 64, _tensor((2048,), torch.uint8), _tensor((32,), torch.float32))
    X8, sx = _tensor((5, 64), torch.int8), _tensor((5,), torch.float32)
    q, k, pos, freq = (_tensor((5, 4, 64), F16), _tensor((5, 2, 64), F16), _tensor((5,), I32),
                       _tensor((32,), torch.int64))
    calls = [lambda: bsp.kv_step(pages, None, far((3,), I32), 8),
             lambda: bsp.kv_step(pages, far((3,), I32), _tensor((3,), I32), 8),
             lambda: bsp.kv_step(pages, None, _tensor((3,), I32), 8, tree_mask=far((8,), torch.int64)),
             lambda: bsp.qk_norm_rope(q, far((5, 2, 64), F16), pos, freq),
             lambda: bsp.qk_norm_rope(q, k, far((5,), I32), freq),
             lambda: bsp.qk_norm_rope(q, k, pos, far((32,), torch.int64)),
             lambda: bsp.qk_norm_rope(q, k, pos, freq, q_weight=far((64,), F16)),
             lambda: bsp.qk_norm_rope_append(q, k, k, pos, freq, _cache(), far((5,), torch.int64)),
             lambda: bsp.qk_norm_rope_append(far((5, 4, 64), F16), k, k, pos, freq, _cache(), _tensor((5,), torch.int64)),
             lambda: bsp.quantize_tokens(_tensor((5, 64), F16), bsp.INT8, weight=far((64,), F16)),
             lambda: bsp.quantize_tokens(_tensor((5, 64), F16), bsp.INT8, residual=far((5, 64), F16)),
             lambda: bsp.dequantize_tokens(far((5, 64), torch.int8), sx, bsp.INT8, 64),
             lambda: bsp.gemm_w8a8(W, far((5, 64), torch.int8), sx),
             lambda: bsp.gemm_w8a8(W, X8, far((5,), torch.float32)),
             lambda: bsp.gemm_w8a8(W, X8, sx, workspace=far((1 << 20,), torch.uint8)),
             lambda: bsp.KVPages(_tensor((3, 4), I32), far((3,), I32), _tensor((3,), I32), _tensor((10,), I32), 16)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
        assert not world.lib.calls, i


def test_shapes_and_types_that_do_not_fit(world):
    W = bsp.DenseInt8(32, 100, _tensor((4096,), torch.uint8), _tensor((32,), torch.float32))
    wide = _tensor((5, 112), torch.int8)
    bsp.gemm_w8a8(W, wide[:, :100], _tensor((5,), torch.float32))
    assert world.lib.calls.pop()[1][4] == 112
    q, k, pos = _tensor((5, 4, 64), F16), _tensor((5, 2, 64), F16), _tensor((5,), I32)
    t = _tensor((5, 64), F16)
    calls = [
        # the last row ends before its stride: the kernel reads whole pieces
        lambda: bsp.gemm_w8a8(W, torch.as_strided(_tensor((4 * 112 + 100,), torch.int8), (5, 100), (112, 1)),
                              _tensor((5,), torch.float32)),
        lambda: bsp.gemm_w8a8(W, _tensor((5, 99), torch.int8), _tensor((5,), torch.float32)),
        lambda: bsp.gemm_w8a8(W, _tensor((5, 100), torch.uint8), _tensor((5,), torch.float32)),
        lambda: bsp.gemm_w8a8(W, wide[:, :100], _tensor((4,), torch.float32)),
        lambda: bsp.gemm_w8a8(W, wide[:, :100], _tensor((5,), torch.float32), Y=_tensor((5, 31), F16)),
        lambda: bsp.quantize_tokens(t, bsp.FP16),
        lambda: bsp.quantize_tokens(t, bsp.INT8, hidden=t),
        lambda: bsp.quantize_tokens(t, bsp.INT8, weight=_tensor((63,), F16)),
        lambda: bsp.quantize_tokens(t, bsp.INT8, codes=_tensor((5, 64), torch.uint8)),
        lambda: bsp.quantize_tokens(t, bsp.INT4, codes=_tensor((5, 31), torch.uint8)),
        lambda: bsp.quantize_tokens(t.t(), bsp.INT8),
        lambda: bsp.dequantize_tokens(_tensor((5, 64), torch.int8), _tensor((5,), torch.float32), bsp.INT2, 64),
        lambda: bsp.qk_norm_rope(q, _tensor((4, 2, 64), F16), pos, None),
        lambda: bsp.qk_norm_rope(q, k, _tensor((4,), I32), _tensor((32,), torch.int64)),
        lambda: bsp.qk_norm_rope(q, k, pos.to(torch.int64), _tensor((32,), torch.int64)),
        lambda: bsp.qk_norm_rope(q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, None),
        lambda: bsp.qk_norm_rope_append(_tensor((5, 4, 128), F16), k, k, pos, None, _cache(), _tensor((5,), torch.int64)),
        lambda: bsp.kv_step(bsp.KVPages(_tensor((3, 4), I32), _tensor((3,), I32), _tensor((3,), I32), _tensor((10,), I32),
                                        16), None, _tensor((4,), I32), 8),
    ]
    for i, call in enumerate(calls):
        with pytest.raises((TypeError, ValueError)):
            call()
        assert not world.lib.calls, i


def test_pages_given_another_storage(world):
    pages = bsp.KVPages(_tensor((3, 4), I32), _tensor((3,), I32), _tensor((3,), I32), _tensor((10,), I32), 16)
    for name, shape in (("block_table", (3, 4)), ("lens", (3,)), ("held", (3,)), ("free", (10,))):
        before = getattr(pages, name).data_ptr()
        getattr(pages, name).data = torch.ones(shape, dtype=I32)
        assert getattr(pages, name).data_ptr() != before
        bsp.kv_step(pages, None, _tensor((3,), I32), 8)
        d = bsp._KVPagesDesc.from_address(world.lib.calls[-1][1][0])
        assert (d.block_table, d.lens, d.held, d.free_pages) == tuple(
            getattr(pages, n).data_ptr() for n in ("block_table", "lens", "held", "free"))
    calls = len(world.lib.calls)
    pages.lens.data = torch.ones(2, dtype=I32)
    with pytest.raises(ValueError):
        bsp.kv_step(pages, None, _tensor((3,), I32), 8)
    assert len(world.lib.calls) == calls


def test_tokens_without_a_channel_are_refused(world):
    with pytest.raises(ValueError):
        bsp.quantize_tokens(_tensor((3, 0), F16), bsp.INT8)
