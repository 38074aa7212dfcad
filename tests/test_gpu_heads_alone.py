"""Query heads without key heads, and key heads without query heads: the kinds a call does not have are not touched,
neither their rows (which have no address) nor the cache's slots."""
import ctypes

import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _heads(rng, n, h, D, dev):
    return torch.from_numpy(rng.normal(0, 1, (n, h, D)).astype(np.float16)).to(dev)


# queries that fill their last wavefront in part (one head, 5, 9), and whole ones; enough of them for two groups a
# wavefront (heads of 128 from 32768 on)
@pytest.mark.parametrize("n,h", [(1, 1), (3, 5), (2, 9), (4, 8), (33, 16), (3700, 9)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_alone(D, n, h, dev):
    rng = np.random.default_rng(D + n + h)
    Q, K = _heads(rng, n, h, D, dev), _heads(rng, n, 2, D, dev)
    none = torch.empty((n, 0, D), dtype=torch.float16, device=dev)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    freq = bsp.rope_frequencies(D, device=dev)
    w = _heads(rng, 1, 1, D, dev).view(D)
    args = dict(q_weight=w, k_weight=w)
    want, _ = bsp.qk_norm_rope(Q, K, pos, freq, **args)
    q, k = bsp.qk_norm_rope(Q, none, pos, freq, **args)
    assert torch.equal(q, want) and k.shape == (n, 0, D)
    for kind in (bsp.FP16, bsp.INT8, bsp.INT4):
        cache = bsp.new_kv_cache(kind, 4, 0, 16, D, device=dev)
        q = bsp.qk_norm_rope_append(Q, none, none, pos, freq, cache, pos.long(), **args)
        assert torch.equal(q, want)
    # the C entries, with nothing where nothing is needed
    d = bsp._rotation(pos, freq, w, w, 1e-6, False, n, D, 0)
    L, stream = bsp.load_library(), torch.cuda.current_stream().cuda_stream
    for call in (lambda o: L.qk_norm_rope_f16(Q.data_ptr(), h * D, None, 0, n, h, 0, D, d, o.data_ptr(), h * D, None, 0, stream),
                 lambda o: L.qk_norm_rope_append_f16(Q.data_ptr(), h * D, None, 0, None, 0, n, h, d,
                                                     ctypes.addressof(cache._desc), None, o.data_ptr(), h * D, stream)):
        o = torch.zeros_like(Q)
        assert call(o) == bsp.OK
        torch.cuda.synchronize()
        assert torch.equal(o, want)


@pytest.mark.parametrize("n,h", [(1, 1), (3, 5), (2, 9), (3700, 9)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_alone(D, n, h, dev):
    rng = np.random.default_rng(D + n + h)
    Q, K, V = (_heads(rng, n, m, D, dev) for m in (2, h, h))
    none = torch.empty((n, 0, D), dtype=torch.float16, device=dev)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    freq = bsp.rope_frequencies(D, device=dev)
    _, want = bsp.qk_norm_rope(Q, K, pos, freq)
    q, k = bsp.qk_norm_rope(none, K, pos, freq)
    assert torch.equal(k, want) and q.shape == (n, 0, D)
    one, two = (bsp.new_kv_cache(bsp.INT8, -(-n // 16), h, 16, D, device=dev) for _ in range(2))
    assert bsp.qk_norm_rope_append(none, K, V, pos, freq, one, pos.long()).shape == (n, 0, D)
    bsp.kv_append(two, want, V, pos.long())
    torch.cuda.synchronize()
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(one, name), getattr(two, name))
