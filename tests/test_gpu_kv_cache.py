"""The quantised paged cache on the GPU against the oracle: codes and scale
words bit for bit, values read back within one fp16 rounding."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import serving

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
KINDS = {"fp16": bsp.FP16, "int8": bsp.INT8, "int4": bsp.INT4}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _rows(rng, n, heads, D):
    """Rows of mixed size, with channel offsets, constants, ties and tiny values among them."""
    x = rng.normal(0, 1, (n, heads, D)) * np.exp(rng.normal(0, 2, (n, heads, 1))) + rng.normal(0, 1, (1, heads, D))
    x = x.astype(np.float16)
    flat = x.reshape(-1, D)
    for i in range(0, flat.shape[0], 7):
        flat[i] = [np.full(D, -3.0), np.arange(D) % 16 * 0.5, np.full(D, 2.0 ** -24) * (np.arange(D) % 3),
                   np.where(np.arange(D) % 2, 65504.0, -65504.0), np.zeros(D)][(i // 7) % 5]
    return x


def _stored(cache, name, slots):
    """(codes, words) at the slots, [n][heads][...]."""
    ps = cache.page_size
    codes = getattr(cache, name).cpu().numpy()[slots // ps, :, slots % ps]
    w = getattr(cache, name + "_scale")
    return codes, None if w is None else w.cpu().numpy().view(np.uint32)[slots // ps, :, slots % ps]


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("n,heads,D,page", [(1, 1, 64, 16), (1, 3, 128, 32), (7, 2, 256, 16), (33, 5, 128, 64),
                                            (130, 1, 64, 16), (257, 2, 128, 128)])
def test_append_and_gather(kind, n, heads, D, page, dev):
    rng = np.random.default_rng(n * 31 + heads + D + page)
    pages = -(-n // page) + 2
    cache = bsp.new_kv_cache(KINDS[kind], pages, heads, page, D, device=dev)
    K, V = _rows(rng, n, heads, D), _rows(rng, n, heads, D)
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    bsp.kv_append(cache, torch.from_numpy(K).to(dev), torch.from_numpy(V).to(dev), torch.from_numpy(slots).to(dev))
    out = bsp.kv_gather(cache, torch.from_numpy(slots).to(dev))
    torch.cuda.synchronize()
    untouched = np.setdiff1d(np.arange(pages * page), slots)
    for name, x, got in (("k", K, out[0]), ("v", V, out[1])):
        codes, words = _stored(cache, name, slots)
        got = got.cpu().numpy()
        if kind == "fp16":
            assert np.array_equal(codes.view(np.uint16), x.view(np.uint16))
            assert np.array_equal(got.view(np.uint16), x.view(np.uint16))
        else:
            wc, ww = serving.quantise(x, kind)
            assert np.array_equal(words, ww) and np.array_equal(codes, wc)
            want = np.minimum(serving.dequantise(wc, ww, kind), 65504.0)      # saturating
            # fp32 sum, then fp16: within half an fp16 step plus the sum's own rounding
            ulp = np.spacing(np.clip(np.abs(want), 2.0 ** -14, 6e4).astype(np.float16)).astype(np.float64)
            assert (np.abs(got.astype(np.float64) - want) <= 0.5 * ulp + np.abs(want) * 2.0 ** -23).all()
        rest, rw = _stored(cache, name, untouched)
        assert not rest.any() and (rw is None or not rw.any()), "a slot of no token was written"


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
def test_slots_outside_the_cache(kind, dev):
    rng = np.random.default_rng(5)
    cache = bsp.new_kv_cache(KINDS[kind], 2, 2, 16, 64, device=dev)
    K, V = _rows(rng, 6, 2, 64), _rows(rng, 6, 2, 64)
    slots = np.array([3, -1, 32, 31, 1 << 40, -(1 << 40)], np.int64)
    s = torch.from_numpy(slots).to(dev)
    bsp.kv_append(cache, torch.from_numpy(K).to(dev), torch.from_numpy(V).to(dev), s)
    k, v = bsp.kv_gather(cache, s)
    torch.cuda.synchronize()
    written = cache.k.cpu().numpy().reshape(2, 2, 16, -1).any((1, 3)).reshape(-1)
    assert np.flatnonzero(written).tolist() == [3, 31]
    for t in (k, v):
        assert not t[[1, 2, 4, 5]].any() and t[[0, 3]].any(dim=-1).all()


def test_strided_and_unaligned_rows(dev):
    # K and V as slices of a fused projection's output, one of them off a 16-byte boundary
    rng = np.random.default_rng(6)
    n, heads, D, hq = 19, 2, 128, 3
    for odd in (0, 1):
        wide = torch.from_numpy(rng.normal(0, 1, (n, (hq + 2 * heads) * D + 8 + odd)).astype(np.float16)).to(dev)
        K = wide[:, hq * D + odd:(hq + heads) * D + odd].view(n, heads, D) if odd == 0 else \
            wide[:, hq * D + odd:(hq + heads) * D + odd].unflatten(1, (heads, D))
        V = wide[:, (hq + heads) * D + odd:(hq + 2 * heads) * D + odd].unflatten(1, (heads, D))
        cache = bsp.new_kv_cache(bsp.INT4, 3, heads, 16, D, device=dev)
        slots = np.arange(5, 5 + n)
        bsp.kv_append(cache, K, V, torch.from_numpy(slots).to(dev))
        out = torch.zeros_like(wide)
        ko = out[:, odd:heads * D + odd].unflatten(1, (heads, D))
        vo = out[:, heads * D + odd:2 * heads * D + odd].unflatten(1, (heads, D))
        bsp.kv_gather(cache, torch.from_numpy(slots).to(dev), K=ko, V=vo)
        k2, v2 = bsp.kv_gather(cache, torch.from_numpy(slots).to(dev))
        torch.cuda.synchronize()
        for name, x in (("k", K), ("v", V)):
            codes, words = _stored(cache, name, slots)
            wc, ww = serving.quantise(x.cpu().numpy(), "int4")
            assert np.array_equal(codes, wc) and np.array_equal(words, ww)
        assert torch.equal(ko, k2) and torch.equal(vo, v2)
        assert not out[:, 2 * heads * D + odd:].any() and not out[:, :odd].any()


def test_infinities_and_nan_mark_their_row_only(dev):
    x = np.random.default_rng(7).normal(0, 1, (3, 2, 64)).astype(np.float16)
    x[0, 0, 63], x[1, 1, 0], x[2, 0, 5] = np.nan, np.inf, -np.inf
    for kind in ("int8", "int4"):
        cache = bsp.new_kv_cache(KINDS[kind], 1, 2, 16, 64, device=dev)
        t, slots = torch.from_numpy(x).to(dev), torch.arange(3, device=dev)
        bsp.kv_append(cache, t, t, slots)
        k, v = bsp.kv_gather(cache, slots)
        codes, words = _stored(cache, "k", np.arange(3))
        wc, ww = serving.quantise(x, kind)
        assert np.array_equal(codes, wc) and np.array_equal(words, ww)
        bad = torch.isnan(k).all(-1).cpu().numpy()
        assert bad.tolist() == [[True, False], [False, True], [True, False]]
        assert torch.isfinite(k.cpu()[~torch.from_numpy(bad)]).all() and torch.equal(k.isnan(), v.isnan())


def test_empty_calls_and_another_stream(dev):
    cache = bsp.new_kv_cache(bsp.INT8, 4, 2, 16, 64, device=dev)
    none = torch.empty((0, 2, 64), dtype=torch.float16, device=dev)
    slots = torch.empty(0, dtype=torch.int64, device=dev)
    bsp.kv_append(cache, none, none, slots)
    assert bsp.kv_gather(cache, slots)[0].shape == (0, 2, 64)
    x = torch.randn(64, 2, 64, device=dev).half()
    slots = torch.arange(64, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bsp.kv_append(cache, x, x, slots, stream=side)
    k, _ = bsp.kv_gather(cache, slots, stream=side)
    torch.cuda.synchronize()
    codes, _ = _stored(cache, "k", np.arange(64))
    assert np.array_equal(codes, serving.quantise(x.cpu().numpy(), "int8")[0])
    assert (k - x).abs().max() < 0.05
