"""The dense 8-bit product on the GPU: exact sums, so equal to the oracle bit for bit."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _problem(rng, N, M, K, dev, pitch=None, extreme=False):
    """W, X (rows `pitch` bytes apart, garbage behind them), scales, on the host; X on the GPU."""
    if extreme:
        W = rng.choice(np.array([-128, 127], np.int8), (M, K))
        x = rng.choice(np.array([-128, 127], np.int8), (N, K))
    else:
        W = rng.integers(-128, 128, (M, K)).astype(np.int8)
        x = rng.integers(-128, 128, (N, K)).astype(np.int8)
    pitch = -(-K // 16) * 16 if pitch is None else pitch
    wide = rng.integers(-128, 128, (N, pitch)).astype(np.int8)
    wide[:, :K] = x
    sw = (rng.random(M) * 0.001 + 0.0001).astype(np.float32)
    sx = (rng.random(N) * 0.01 + 0.001).astype(np.float32)
    return W, x, torch.from_numpy(wide).to(dev)[:, :K], sw, sx


def _run(W, X, sw, sx, dev, workspace=True, **kw):
    enc = bsp.encode_int8(W, sw).to_device(dev)
    ws = bsp.new_gemm_workspace(enc, X.shape[0], device=dev) if workspace else None
    return bsp.gemm_w8a8(enc, X, torch.from_numpy(sx).to(dev), workspace=ws, **kw)


def _same(Y, want):
    assert np.array_equal(Y.cpu().numpy().view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("N,M,K", [
    (1, 1, 1), (1, 16, 64), (1, 17, 65), (2, 100, 1001), (3, 333, 127), (8, 64, 4096), (16, 48, 640), (17, 48, 640),
    (31, 1000, 250), (32, 512, 1024), (33, 512, 1024), (48, 130, 515), (64, 256, 512), (65, 257, 513), (100, 1008, 96),
    (127, 128, 128), (128, 128, 128), (129, 129, 129), (200, 64, 2000), (255, 300, 77), (256, 256, 256), (257, 255, 1025),
    (300, 4100, 200), (513, 700, 640), (1000, 1000, 1000), (1, 4096, 4096), (32, 4096, 11008), (4, 20000, 64), (5, 16, 40000)])
def test_sizes(N, M, K, workspace, dev):
    rng = np.random.default_rng(N * 3 + M * 5 + K)
    W, x, X, sw, sx = _problem(rng, N, M, K, dev)
    _same(_run(W, X, sw, sx, dev, workspace), step.product(W, x, sw, sx))


@pytest.mark.parametrize("N", [1, 20, 70, 300])
def test_largest_sums(N, dev):
    # all products of one sign at the largest K: sums next to 2^31
    K, M = 131071, 33
    W = np.full((M, K), -128, np.int8)
    W[::2] = 127
    x = np.full((N, K), -128, np.int8)
    x[::3] = 127
    X = torch.zeros((N, K + 1), dtype=torch.int8, device=dev)
    X[:, :K] = torch.from_numpy(x).to(dev)
    sw, sx = np.full(M, 2.0 ** -10, np.float32), np.full(N, 2.0 ** -8, np.float32)
    _same(_run(W, X[:, :K], sw, sx, dev), step.product(W, x, sw, sx))


@pytest.mark.parametrize("N", [1, 9, 40, 150, 400])
@pytest.mark.parametrize("K,pitch", [(100, 112), (100, 256), (64, 80), (1000, 1008), (1000, 4096)])
def test_row_strides_and_what_lies_past_a_row(N, K, pitch, dev):
    rng = np.random.default_rng(N + K + pitch)
    M = 200
    W, x, X, sw, sx = _problem(rng, N, M, K, dev, pitch, extreme=True)
    wide = torch.full((N, M + 9), 5.0, dtype=torch.float16, device=dev)
    _run(W, X, sw, sx, dev, Y=wide[:, 3:3 + M])
    torch.cuda.synchronize()
    _same(wide[:, 3:3 + M].contiguous(), step.product(W, x, sw, sx))
    assert (wide[:, :3] == 5).all() and (wide[:, 3 + M:] == 5).all()


def test_scales_that_are_not_finite_reach_their_row_and_column_only(dev):
    rng = np.random.default_rng(6)
    W, x, X, sw, sx = _problem(rng, 37, 90, 128, dev)
    sw[5], sx[7], sx[20] = np.nan, np.nan, np.inf
    with np.errstate(invalid="ignore"):
        want = step.product(W, x, sw, sx)
    got = _run(W, X, sw, sx, dev).cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_empty_calls(dev):
    enc = bsp.encode_int8(np.zeros((5, 64), np.int8), np.ones(5, np.float32)).to_device(dev)
    none = torch.empty((0, 64), dtype=torch.int8, device=dev)
    assert bsp.gemm_w8a8(enc, none, torch.empty(0, device=dev)).shape == (0, 5)
    enc = bsp.encode_int8(np.zeros((5, 0), np.int8), np.ones(5, np.float32)).to_device(dev)
    X = torch.empty((3, 0), dtype=torch.int8, device=dev)
    Y = torch.full((3, 5), 7.0, dtype=torch.float16, device=dev)
    bsp.gemm_w8a8(enc, X, torch.ones(3, device=dev), Y=Y)
    assert not Y.any()
    enc = bsp.encode_int8(np.zeros((0, 64), np.int8), np.ones(0, np.float32)).to_device(dev)
    assert bsp.gemm_w8a8(enc, torch.zeros((2, 64), dtype=torch.int8, device=dev), torch.ones(2, device=dev)).shape == (2, 0)


@pytest.mark.parametrize("N,M,K", [(1, 4096, 4096), (48, 1024, 4096), (140, 512, 11008)])
def test_streams_graph_and_one_workspace(N, M, K, dev):
    rng = np.random.default_rng(N)
    W, x, X, sw, sx = _problem(rng, N, M, K, dev)
    want = step.product(W, x, sw, sx)
    enc = bsp.encode_int8(W, sw).to_device(dev)
    s = torch.from_numpy(sx).to(dev)
    ws = torch.zeros(max(1 << 20, bsp.gemm_workspace_bytes(M, K, N)), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y = bsp.gemm_w8a8(enc, X, s, workspace=ws, stream=side)
    torch.cuda.synchronize()
    _same(Y, want)
    out, second = torch.zeros_like(Y), torch.zeros_like(Y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsp.gemm_w8a8(enc, X, s, Y=out, workspace=ws)
        bsp.gemm_w8a8(enc, X, s, Y=second, workspace=ws)
    for k in range(4):
        out.zero_(), second.zero_()
        X.copy_(torch.from_numpy(rng.integers(-128, 128, (N, K)).astype(np.int8)).to(dev))
        graph.replay()
        eager = bsp.gemm_w8a8(enc, X, s, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(second, eager)
        _same(out, step.product(W, X.cpu().numpy(), sw, sx))


def test_tokens_into_the_product(dev):
    rng = np.random.default_rng(21)
    for N, M, K in ((1, 64, 100), (50, 300, 1000)):
        X16 = rng.normal(0, 1, (N, K)).astype(np.float16)
        W = rng.integers(-127, 128, (M, K)).astype(np.int8)
        sw = (rng.random(M) * 0.001 + 0.0001).astype(np.float32)
        t = bsp.quantize_tokens(torch.from_numpy(X16).to(dev), bsp.INT8)
        enc = bsp.encode_int8(W, sw).to_device(dev)
        Y = bsp.gemm_w8a8(enc, t.codes, t.scale)
        codes, _, _, _ = step.quantise_tokens(X16, 127)
        _same(Y, step.product(W, codes, sw, t.scale.cpu().numpy()))


def test_one_workspace_for_fewer_tokens(dev):
    rng = np.random.default_rng(31)
    M, K, most = 512, 11008, 1200
    W, x, X, sw, sx = _problem(rng, most, M, K, dev)
    enc = bsp.encode_int8(W, sw).to_device(dev)
    ws = bsp.new_gemm_workspace(enc, most, device=dev)
    s, want = torch.from_numpy(sx).to(dev), step.product(W, x, sw, sx)
    for N in (most, 1, 600, 16, 1025, 897, 33, most):
        _same(bsp.gemm_w8a8(enc, X[:N], s[:N], workspace=ws), want[:N])


def test_more_tokens_than_one_launch_takes(dev):
    # one channel: 2^22 - 8 tiles of 16 tokens a launch
    N, K = ((1 << 22) - 8) * 16 + 33, 16
    g = torch.Generator(device=dev).manual_seed(5)
    X = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=dev, generator=g)
    w = np.arange(-120, 120, 15, dtype=np.int8).reshape(1, K)
    sx = torch.rand(N, device=dev, generator=g) * 0.001
    Y = bsp.gemm_w8a8(bsp.encode_int8(w, np.full(1, 0.5, np.float32)).to_device(dev), X, sx)
    sums = torch.zeros(N, device=dev)      # whole numbers below 2^24: exact
    for k in range(K):
        sums += X[:, k].float() * float(w[0, k])
    assert torch.equal(Y[:, 0], (sums * 0.5 * sx).half())


@pytest.mark.parametrize("N", [3, 8, 16])
def test_weights_past_the_last_level_cache(N, dev):
    rng = np.random.default_rng(N)
    M, K = 25700, 4100      # over 96 MB
    W, x, X, sw, sx = _problem(rng, N, M, K, dev)
    Y = _run(W, X, sw, sx, dev)
    rows = rng.permutation(M)[:300]
    rows[:2] = 0, M - 1
    assert np.array_equal(Y.cpu().numpy()[:, rows].view(np.uint16), step.product(W[rows], x, sw[rows], sx).view(np.uint16))
