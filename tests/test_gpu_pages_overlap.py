"""Results and inputs of a step in one allocation, side by side; and the lengths themselves as what is kept."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


@pytest.mark.parametrize("B,rows", [(3, 10), (300, 3000)])
def test_side_by_side(B, rows, dev):
    rng = np.random.default_rng(B)
    new = torch.from_numpy(rng.integers(0, 10, B).astype(np.int32)).to(dev)
    lens = torch.from_numpy(rng.integers(0, 40, B).astype(np.int32)).to(dev)

    def pages():
        p = bsp.new_kv_pages(B, 4, 4 * B, 16, device=dev)
        bsp.kv_step(p, None, lens, 40 * B)
        return p

    want = bsp.kv_step(pages(), lens, new, rows)
    sizes = [2 * rows, rows, rows, B + 1 + (B + 1) % 2, B + B % 2, B, B]
    parts = torch.split(torch.zeros(sum(sizes), dtype=torch.int32, device=dev), sizes)
    out = bsp.KVStep(parts[0].view(torch.int64), parts[1], parts[2], parts[3][:B + 1], parts[4][:B])
    parts[5].copy_(lens), parts[6].copy_(new)
    p = pages()
    bsp.kv_step(p, parts[5], parts[6], rows, out=out)
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    # the lengths themselves, which the call updates
    q = pages()
    got = bsp.kv_step(q, q.lens, new, rows)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(p.lens, q.lens) and torch.equal(p.free, q.free)
    with pytest.raises(bsp.BspError) as e:
        bsp.kv_step(q, got.kv_lens, new, rows, out=got)
    assert e.value.status == bsp.E_ARG
    bsp.kv_step(q, got.kv_lens, new, rows)
