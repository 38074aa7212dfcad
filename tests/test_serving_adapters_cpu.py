"""Adapters whose tensors get another storage between calls: the call goes to
what the tensors hold then. Shown without a GPU, with tensors that claim to lie
on one and a library that launches nothing."""
import pytest

import bit_unstructured_sparse_amd as bsp
from test_serving_streams_cpu import World, _matrix, _tensor

torch = pytest.importorskip("torch")


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def _call(ad, M=64, K=128):
    return bsp.spmm_f16_lora(_matrix(bsp.FP16, M, K), _tensor((8, K), torch.float16), ad, _tensor((8,), torch.int32))


@pytest.mark.parametrize("name,shape,dtype", [("A", (2, 16, 128), torch.float16), ("B", (2, 64, 16), torch.float16),
                                              ("scale", (2,), torch.float32), ("rank", (2,), torch.int32)])
def test_a_new_storage_is_used(name, shape, dtype, world):
    ad = bsp.LoraAdapters(_tensor((2, 16, 128), torch.float16), _tensor((2, 64, 16), torch.float16),
                          _tensor((2,), torch.float32), _tensor((2,), torch.int32))
    _call(ad)
    before = getattr(ad, name).data_ptr()
    getattr(ad, name).data = torch.ones(shape, dtype=dtype)
    assert getattr(ad, name).data_ptr() != before
    _call(ad)
    d = world.lib.calls[-1][1][8]._obj
    field = {"A": d.A, "B": d.B, "scale": d.scale, "rank": d.ranks}[name]
    assert field == getattr(ad, name).data_ptr()


def test_a_new_storage_of_another_shape_is_refused(world):
    ad = bsp.LoraAdapters(_tensor((2, 16, 128), torch.float16), _tensor((2, 64, 16), torch.float16))
    _call(ad)
    ad.A.data = torch.ones((2, 8, 128), dtype=torch.float16)      # the rank of A and of B differ
    with pytest.raises(ValueError):
        _call(ad)
    ad.B.data = torch.ones((2, 64, 8), dtype=torch.float16)
    _call(ad)
    assert world.lib.calls[-1][1][8]._obj.rank == 8
    ad.A.data = torch.ones((2, 8, 64), dtype=torch.float16)       # another K
    with pytest.raises(ValueError):
        _call(ad)
    assert len(world.lib.calls) == 2
