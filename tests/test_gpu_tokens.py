"""Token quantisation on the GPU against the oracle: codes and sums bit for bit, scales
within the rounding of their fp32 sums."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
LEVELS = {bsp.INT8: 127, bsp.INT4: 7}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _rows(rng, n, K):
    """Rows of mixed size, with constants, ties between codes, zeros and tiny values among them."""
    x = rng.normal(0, 1, (n, K)) * np.exp(rng.normal(0, 2, (n, 1)))
    x = x.astype(np.float16)
    for i in range(0, n, 5):
        half = (np.arange(K) % 255 - 127) * 0.5          # halves of the largest over 127: ties, both signs
        tie = np.where(np.arange(K) == K // 2, 127.0, half)
        x[i] = [tie, np.full(K, -3.0), np.zeros(K), np.full(K, 2.0 ** -24) * (np.arange(K) % 3),
                np.where(np.arange(K) % 2, 65504.0, -65504.0)][(i // 5) % 5]
    return x


def _unpacked(t, dtype, K):
    c = t.codes.cpu().numpy()
    if dtype == bsp.INT8:
        return c.astype(np.int64)
    c = np.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)[:, :K].astype(np.int64)
    return np.where(c >= 8, c - 16, c)


def check(t, X, dtype, weight, eps, residual, dev):
    codes, scale, x16, h = step.quantise_tokens(X, LEVELS[dtype], weight, eps, residual)
    assert np.array_equal(_unpacked(t, dtype, X.shape[1]), codes)
    if dtype == bsp.INT4:
        assert np.array_equal(t.codes.cpu().numpy(), step.pack_int4(codes))
    got = t.scale.cpu().numpy().astype(np.float64)
    # a lane's chain of fma (32 at most where registers hold the row, K / 4096 past that), 6 + 8 additions across lanes
    # and wavefronts, halved by the root, then a division, a root, a product and a division
    steps = (max(32, X.shape[1] // 512) + 14) / 2 + 5
    assert np.array_equal(np.isnan(got), np.isnan(scale))
    assert (np.abs(got - scale)[~np.isnan(scale)] <= (scale * steps * 2.0 ** -24 + 2.0 ** -149)[~np.isnan(scale)]).all()
    if t.hidden is not None:
        assert np.array_equal(t.hidden.cpu().numpy().view(np.uint16), h.view(np.uint16))
    if t.x16 is not None:
        fine = np.isfinite(x16) & (np.abs(x16) < 65000)
        err = np.abs(t.x16.cpu().numpy().astype(np.float64) - x16)
        assert (err <= np.abs(x16) * (2.0 ** -11 + steps * 2.0 ** -24) + 2.0 ** -25)[fine].all()


@pytest.mark.parametrize("dtype", [bsp.INT8, bsp.INT4])
@pytest.mark.parametrize("n,K", [(1, 1), (3, 7), (1, 64), (5, 100), (9, 512), (2, 513), (7, 1001), (4, 2048), (3, 4096),
                                 (30, 4104), (2, 8192), (2, 8193), (3, 12271), (2, 16384), (1, 16385), (2, 20000)])
@pytest.mark.parametrize("norm,res,want", [(False, False, False), (True, True, True), (True, False, False),
                                           (False, True, False)])
def test_codes_scales_sums(dtype, n, K, norm, res, want, dev):
    rng = np.random.default_rng(n * 7 + K + dtype)
    X = _rows(rng, n, K)
    weight = (1 + 0.2 * rng.normal(0, 1, K)).astype(np.float16) if norm else None
    residual = rng.normal(0, 2, (n, K)).astype(np.float16) if res else None
    on = lambda a: None if a is None else torch.from_numpy(a).to(dev)
    t = bsp.quantize_tokens(on(X), dtype, weight=on(weight), eps=1e-5, residual=on(residual), x16=want)
    torch.cuda.synchronize()
    check(t, X, dtype, weight, 1e-5, residual, dev)
    # reading back: the fp32 product, rounded once
    back = bsp.dequantize_tokens(t.codes, t.scale, dtype, K).cpu().numpy()
    with np.errstate(over="ignore"):
        expect = (_unpacked(t, dtype, K).astype(np.float32) * t.scale.cpu().numpy()[:, None]).astype(np.float16)
    assert np.array_equal(back, expect)


@pytest.mark.parametrize("dtype", [bsp.INT8, bsp.INT4])
@pytest.mark.parametrize("K,off", [(512, 0), (512, 8), (512, 1), (4096, 3), (333, 0), (10, 2)])
def test_strided_rows_and_sums_in_place(dtype, K, off, dev):
    # columns of a wider tensor, some off a 16-byte boundary; what lies beside them stays
    rng = np.random.default_rng(K + off)
    n, pitch = 11, K + 40
    wide = torch.from_numpy(_rows(rng, n, pitch)).to(dev)
    X = wide[:, off:off + K]
    res = torch.from_numpy(rng.normal(0, 2, (n, pitch)).astype(np.float16)).to(dev)
    R = res[:, off:off + K]
    weight = torch.from_numpy((1 + 0.2 * rng.normal(0, 1, K)).astype(np.float16)).to(dev)
    x, r = X.cpu().numpy(), R.cpu().numpy()
    bytes_ = K if dtype == bsp.INT8 else (K + 1) // 2
    store = torch.full((n, bytes_ + 37), 99, dtype=torch.int8 if dtype == bsp.INT8 else torch.uint8, device=dev)
    before = res.clone()
    t = bsp.quantize_tokens(X, dtype, weight=weight, eps=1e-6, residual=R, hidden=R, codes=store[:, :bytes_])
    torch.cuda.synchronize()
    check(t, x, dtype, weight.cpu().numpy(), 1e-6, r, dev)
    keep = torch.ones(pitch, dtype=torch.bool, device=dev)
    keep[off:off + K] = False
    assert torch.equal(res[:, keep], before[:, keep])
    assert (store[:, bytes_:] == 99).all()
    back = torch.zeros((n, pitch), dtype=torch.float16, device=dev)
    bsp.dequantize_tokens(t.codes, t.scale, dtype, K, X=back[:, off:off + K])
    assert torch.equal(back[:, off:off + K], bsp.dequantize_tokens(t.codes, t.scale, dtype, K))
    assert not back[:, keep].any()


@pytest.mark.parametrize("dtype", [bsp.INT8, bsp.INT4])
def test_infinities_and_nan_mark_their_token_only(dtype, dev):
    rng = np.random.default_rng(3)
    for K in (100, 1000, 20000):
        X = rng.normal(0, 1, (6, K)).astype(np.float16)
        X[0, 5], X[2, K - 1], X[3, 0] = np.nan, np.inf, -np.inf
        res = rng.normal(0, 1, X.shape).astype(np.float16)
        X[4, 7], res[4, 7] = 65504, 65504             # the sum passes fp16
        w = np.ones(K, np.float16)
        t = bsp.quantize_tokens(torch.from_numpy(X).to(dev), dtype, weight=torch.from_numpy(w).to(dev), eps=1e-5,
                                residual=torch.from_numpy(res).to(dev))
        assert torch.isnan(t.scale).tolist() == [True, False, True, True, True, False]
        codes, _, _, h = step.quantise_tokens(X, LEVELS[dtype], w, 1e-5, res)
        assert np.array_equal(_unpacked(t, dtype, K), codes) and not codes[[0, 2, 3, 4]].any()
        back = bsp.dequantize_tokens(t.codes, t.scale, dtype, K)
        assert torch.isnan(back).all(-1).tolist() == torch.isnan(t.scale).tolist()
        got = t.hidden.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(h)) and np.array_equal(got[~np.isnan(h)], h[~np.isnan(h)])


def test_zero_tokens_and_no_epsilon(dev):
    X = torch.zeros(3, 64, dtype=torch.float16, device=dev)
    X[1] = 2.0
    w = torch.ones(64, dtype=torch.float16, device=dev)
    t = bsp.quantize_tokens(X, bsp.INT8, weight=w, eps=0.0, x16=True)
    assert not t.codes[[0, 2]].any() and t.scale[[0, 2]].tolist() == [0, 0] and not t.x16[[0, 2]].any()
    assert (t.codes[1] == 127).all() and (t.x16[1] == 1).all()


def test_against_the_host_packer_and_the_sparse_product(dev):
    # what spmm_w4a4_dq takes, without a way through the host
    rng = np.random.default_rng(4)
    n, K, M = 5, 333, 96
    X = rng.normal(0, 1, (n, K)).astype(np.float16)
    t = bsp.quantize_tokens(torch.from_numpy(X).to(dev), bsp.INT4)
    codes, scale, _, _ = step.quantise_tokens(X, 7)
    assert np.array_equal(t.codes.cpu().numpy(), bsp.pack_int4(codes.astype(np.int8)))
    W = (rng.integers(-8, 8, (M, K)) * (rng.random((M, K)) < 0.5)).astype(np.int8)
    sw = rng.random(M).astype(np.float32)
    Y = bsp.spmm_bitmap_w4a4_dq(bsp.encode(W).to_device(dev), t.codes, n, torch.from_numpy(sw).to(dev), t.scale)
    want = step.product(W, codes, sw, t.scale.cpu().numpy())
    assert np.array_equal(Y.cpu().numpy(), want)


def test_streams_and_graph(dev):
    g = torch.Generator(device=dev).manual_seed(5)
    X = torch.randn(33, 1000, generator=g, device=dev).half()
    w = torch.ones(1000, dtype=torch.float16, device=dev)
    res = torch.randn(33, 1000, generator=g, device=dev).half()
    ref = bsp.quantize_tokens(X, bsp.INT8, weight=w, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t = bsp.quantize_tokens(X, bsp.INT8, weight=w, residual=res, stream=side)
    back = bsp.dequantize_tokens(t.codes, t.scale, bsp.INT8, 1000, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(t, ref):
        assert (a is None and b is None) or torch.equal(a, b)
    codes, scale = torch.empty_like(t.codes), torch.empty_like(t.scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsp.quantize_tokens(X, bsp.INT8, weight=w, codes=codes, scale=scale)
        bsp.dequantize_tokens(codes, scale, bsp.INT8, 1000, X=back)
    for seed in range(3):
        X.copy_(torch.randn(33, 1000, generator=g, device=dev).half())
        graph.replay()
        now = bsp.quantize_tokens(X, bsp.INT8, weight=w)
        torch.cuda.synchronize()
        assert torch.equal(codes, now.codes) and torch.equal(scale, now.scale)
        assert torch.equal(back, bsp.dequantize_tokens(now.codes, now.scale, bsp.INT8, 1000))


def test_empty_calls(dev):
    none = torch.empty((0, 64), dtype=torch.float16, device=dev)
    t = bsp.quantize_tokens(none, bsp.INT4)
    assert t.codes.shape == (0, 32) and t.scale.shape == (0,)
    assert bsp.dequantize_tokens(t.codes, t.scale, bsp.INT4, 64).shape == (0, 64)


@pytest.mark.parametrize("dtype", [bsp.INT8, bsp.INT4])
@pytest.mark.parametrize("K", [100, 129, 164, 256, 257, 300, 511, 513])
def test_many_short_tokens(dtype, K, dev):
    # as many as change how a token is spread over lanes: the same codes as in short calls, and the oracle's
    rng = np.random.default_rng(K)
    n = 16390
    X = np.tile(_rows(rng, 1639, K), (10, 1))
    weight = (1 + 0.2 * rng.normal(0, 1, K)).astype(np.float16)
    x, w = torch.from_numpy(X).to(dev), torch.from_numpy(weight).to(dev)
    t = bsp.quantize_tokens(x, dtype, weight=w, eps=1e-5, residual=x)
    for i in range(0, n, 1490):
        s = bsp.quantize_tokens(x[i:i + 1490], dtype, weight=w, eps=1e-5, residual=x[i:i + 1490])
        assert torch.equal(t.codes[i:i + 1490], s.codes) and torch.equal(t.hidden[i:i + 1490].isnan(), s.hidden.isnan())
    last = bsp.Tokens(t.codes[-60:], t.scale[-60:], None, t.hidden[-60:])
    check(last, X[-60:], dtype, weight, 1e-5, X[-60:], dev)
