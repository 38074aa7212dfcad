"""Calls through the native launch: numbers of another kind are refused as ctypes refuses them."""
import ctypes

import pytest

import bit_unstructured_sparse_amd as bsp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    bsp._use_native()
    return torch.device("cuda:0")


@pytest.mark.parametrize("bad", [2.0, None, "2"])
def test_a_number_of_another_kind_is_refused(bad, dev):
    cache = bsp.new_kv_cache(bsp.FP16, 2, 1, 16, 64, device=dev)
    Q = torch.ones(2, 1, 64, dtype=torch.float16, device=dev)
    table, lens = (torch.zeros(1, n, dtype=torch.int32, device=dev) for n in (2, 1))
    start = torch.tensor([0, 2], dtype=torch.int32, device=dev)
    O = torch.full_like(Q, 5.0)
    with pytest.raises((ctypes.ArgumentError, TypeError)):
        bsp.attention_tree(Q, cache, table, lens.view(1), start, bad, O=O)
    pages = bsp.new_kv_pages(1, 2, 4, 16, device=dev)
    out = bsp.kv_step(pages, None, lens.view(1) + 2, 2)
    with pytest.raises((ctypes.ArgumentError, TypeError, ValueError)):
        bsp.kv_step(pages, None, lens.view(1), bad, out=out)
    torch.cuda.synchronize()
    assert (O == 5).all() and pages.lens.tolist() == [2]
