"""Rows far apart, and far into a cache: every offset past 2^32 bytes."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step
from test_gpu_tokens import _rows, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", [bsp.FP16, bsp.INT8, bsp.INT4])
def test_heads_far_into_the_cache(kind, dev):
    rng = np.random.default_rng(kind)
    hkv, D, page = 8, 128, 16
    row = {bsp.FP16: 2 * D, bsp.INT8: D, bsp.INT4: D // 2}[kind]
    pages = (5 << 30) // (hkv * page * row)
    cache = bsp.new_kv_cache(kind, pages, hkv, page, D, device=dev)
    n = 9
    Q, K, V = (torch.from_numpy(rng.normal(0, 1, (n, h, D)).astype(np.float16)).to(dev) for h in (16, hkv, hkv))
    slots = torch.tensor([pages * page - 1, 0, pages * page - 17, pages * page // 2 + 3, 5, pages * page, -1,
                          (1 << 32) // (hkv * row) // page * page + 2, pages * page - 100], device=dev)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    freq = bsp.rope_frequencies(D, device=dev)
    bsp.qk_norm_rope_append(Q, K, V, pos, freq, cache, slots)
    _, k = bsp.qk_norm_rope(Q, K, pos, freq)
    near = bsp.new_kv_cache(kind, 1, hkv, page, D, device=dev)
    bsp.kv_append(near, k, V, pos.long())
    for t, s in enumerate(slots.tolist()):
        if not 0 <= s < pages * page:
            continue
        for name in ("k", "v", "k_scale", "v_scale"):
            far, here = getattr(cache, name), getattr(near, name)
            if far is not None:
                assert torch.equal(far[s // page, :, s % page], here[0, :, t]), (t, name)
    a, b = bsp.kv_gather(cache, slots), bsp.kv_gather(near, pos.long())
    inside = (slots >= 0) & (slots < pages * page)
    assert torch.equal(a[0][inside], b[0][inside]) and torch.equal(a[1][inside], b[1][inside])
    assert not a[0][~inside].any()


def _far(n, width, stride, dev):
    """float16 [n][width], rows `stride` elements apart."""
    return torch.empty((n - 1) * stride + width, dtype=torch.float16, device=dev).as_strided((n, width), (stride, 1))


def test_heads_far_apart(dev):
    rng = np.random.default_rng(3)
    n, hq, hkv, D, stride = 6, 5, 2, 64, (1 << 30) + 8
    x = torch.from_numpy(rng.normal(0, 1, (n, hq + hkv, D)).astype(np.float16)).to(dev)
    far, out = _far(n, (hq + hkv) * D, stride, dev), _far(n, (hq + hkv) * D, stride, dev)
    far.copy_(x.view(n, -1))
    cut = lambda t, a, h: t[:, a * D:(a + h) * D].unflatten(1, (h, D))
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    freq = bsp.rope_frequencies(D, device=dev)
    q, k = bsp.qk_norm_rope(x[:, :hq], x[:, hq:], pos, freq)
    bsp.qk_norm_rope(cut(far, 0, hq), cut(far, hq, hkv), pos, freq, Qo=cut(out, 0, hq), Ko=cut(out, hq, hkv))
    assert torch.equal(cut(out, 0, hq), q) and torch.equal(cut(out, hq, hkv), k)


@pytest.mark.parametrize("dtype", [bsp.INT8, bsp.INT4])
@pytest.mark.parametrize("K", [100, 20001])
def test_tokens_far_apart_and_their_sum_in_place(dtype, K, dev):
    # 20001 channels are read twice: the sum takes its inputs' place as the codes are made
    rng = np.random.default_rng(K)
    n, stride = 7, (1 << 30) + 3
    X, R = _rows(rng, n, K), rng.normal(0, 2, (n, K)).astype(np.float16)
    weight = (1 + 0.2 * rng.normal(0, 1, K)).astype(np.float16)
    w = torch.from_numpy(weight).to(dev)
    x, r = _far(n, K, stride, dev), _far(n, K, stride, dev)
    for into in ("X", "residual"):
        x.copy_(torch.from_numpy(X)), r.copy_(torch.from_numpy(R))
        t = bsp.quantize_tokens(x, dtype, weight=w, eps=1e-5, residual=r, hidden=x if into == "X" else r, x16=True)
        check(t, X, dtype, weight, 1e-5, R, dev)
        other, was = (r, R) if into == "X" else (x, X)
        assert np.array_equal(other.cpu().numpy().view(np.uint16), was.view(np.uint16))
        bsp.dequantize_tokens(t.codes, t.scale, dtype, K, X=other)
        assert torch.equal(other, bsp.dequantize_tokens(t.codes, t.scale, dtype, K))


@pytest.mark.parametrize("N,M,K", [(700, 40, 1000), (2, 40, 1000), (700, 700, 70)])
def test_product_far_apart(N, M, K, dev):
    # the widest rows of X there can be, and results as far apart
    rng = np.random.default_rng(N + M)
    xs, ys = (1 << 23) - 16, 5 << 20
    W, x = rng.integers(-128, 128, (M, K)).astype(np.int8), rng.integers(-128, 128, (N, K)).astype(np.int8)
    X = torch.empty(N * xs, dtype=torch.int8, device=dev).view(N, xs)[:, :K]
    X.copy_(torch.from_numpy(x))
    Y = _far(N, M, ys, dev)
    sw, sx = np.full(M, 0.001, np.float32), (rng.random(N) * 0.01).astype(np.float32)
    enc = bsp.encode_int8(W, sw).to_device(dev)
    bsp.gemm_w8a8(enc, X, torch.from_numpy(sx).to(dev), Y=Y, workspace=bsp.new_gemm_workspace(enc, N, dev))
    assert np.array_equal(Y.cpu().numpy().view(np.uint16), step.product(W, x, sw, sx).view(np.uint16))
