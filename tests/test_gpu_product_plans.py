"""The dense product through every kernel of its plans, equal to the oracle bit for bit, what lies beside its results
untouched."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step
from product_plans import COLUMNS, ONE, SPLIT, STREAM

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _check(N, M, K, workspace, dev, again=1):
    rng = np.random.default_rng(N * 3 + M * 5 + K)
    W = rng.integers(-128, 128, (M, K)).astype(np.int8)
    wide = rng.integers(-128, 128, (N, -(-K // 16) * 16 + 16)).astype(np.int8)      # garbage past K
    sw = (rng.random(M) * 0.001 + 0.0001).astype(np.float32)
    sx = (rng.random(N) * 0.01 + 0.001).astype(np.float32)
    enc = bsp.encode_int8(W, sw).to_device(dev)
    X, s = torch.from_numpy(wide).to(dev)[:, :K], torch.from_numpy(sx).to(dev)
    ws = bsp.new_gemm_workspace(enc, N, device=dev) if workspace else None
    want = step.product(W, wide[:, :K], sw, sx)
    for _ in range(again):
        Y = torch.full((N + 2, M + 5), 5.0, dtype=torch.float16, device=dev)
        bsp.gemm_w8a8(enc, X, s, Y=Y[1:-1, 3:3 + M], workspace=ws)
        got = Y.cpu().numpy()
        assert np.array_equal(got[1:-1, 3:3 + M].view(np.uint16), want.view(np.uint16))
        assert (got[[0, -1]] == 5).all() and (got[:, :3] == 5).all() and (got[:, 3 + M:] == 5).all()
    if ws is not None:
        assert not ws[:65536].any()      # its counters, as they were


@pytest.mark.parametrize("N,M", ONE)
@pytest.mark.parametrize("K", COLUMNS)
def test_whole(N, M, K, dev):
    _check(N, M, K, False, dev)


@pytest.mark.parametrize("N,M,K", SPLIT)
def test_split(N, M, K, dev):
    # twice: the second call finds what the first left in the workspace
    _check(N, M, K, True, dev, again=2)
    _check(N, M, K, False, dev)


@pytest.mark.parametrize("N,M,K", STREAM)
def test_stream(N, M, K, dev):
    _check(N, M, K, False, dev)


def test_largest_sums_in_the_largest_tiles(dev):
    # every product 2^14 at the largest K: sums of 2^31 - 2^14, whole and in parts
    K, M, N = 131071, 300, 520
    W, X = torch.full((M, K), -128, dtype=torch.int8), torch.full((N, K + 1), -128, dtype=torch.int8, device=dev)
    enc = bsp.encode_int8(W.numpy(), np.full(M, 2.0 ** -16, np.float32)).to_device(dev)
    sx = torch.full((N,), 1.0, device=dev)
    want = np.float16(np.float32(K * 2 ** 14) * np.float32(2.0 ** -16))
    for ws in (None, bsp.new_gemm_workspace(enc, N, device=dev)):
        Y = bsp.gemm_w8a8(enc, X[:, :K], sx, workspace=ws)
        assert (Y == float(want)).all()


def test_large_tiles_captured_and_replayed(dev):
    rng = np.random.default_rng(3)
    for N, M, K in ((5480, 73, 130), (1415, 5434, 64)):
        W = rng.integers(-128, 128, (M, K)).astype(np.int8)
        x = rng.integers(-128, 128, (N, -(-K // 16) * 16)).astype(np.int8)
        enc = bsp.encode_int8(W, np.full(M, 0.001, np.float32)).to_device(dev)
        X, s = torch.from_numpy(x).to(dev)[:, :K], torch.full((N,), 0.01, device=dev)
        Y = torch.zeros(N, M, dtype=torch.float16, device=dev)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bsp.gemm_w8a8(enc, X, s, Y=Y)
        for _ in range(3):
            Y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert np.array_equal(Y.cpu().numpy(), step.product(W, x[:, :K], np.full(M, 0.001), np.full(N, 0.01)))
