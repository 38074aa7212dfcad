"""Adapters beside a shared sparse projection on the GPU, against the oracle in
64 bits."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
import workloads
from oracle import serving

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _adapters(rng, n, R, M, K, ranks=None):
    A = (rng.normal(0, 1, (n, R, K)) / np.sqrt(max(K, 1))).astype(np.float16)
    B = (0.3 * rng.normal(0, 1, (n, M, R))).astype(np.float16)
    if ranks is not None:                       # what lies past an adapter's rank is not used
        for a, r in enumerate(ranks):
            A[a, max(r, 0):], B[a, :, max(r, 0):] = np.nan, np.inf
    return A, B, rng.uniform(0.5, 2.0, n).astype(np.float32)


def _dev(dev, A, B, scale, ranks):
    t = lambda x: None if x is None else torch.from_numpy(np.asarray(x)).to(dev)
    return bsp.LoraAdapters(t(A), t(B), t(scale), t(None if ranks is None else np.asarray(ranks, np.int32)))


def _bound(want, base_abs, X, A, B, index, scale, ranks, K):
    """The result's rounding, and fp32 sums: K products of the projection (their
    order free), K and R of the adapter."""
    z = lambda x: np.nan_to_num(np.abs(x.astype(np.float64)), nan=0.0, posinf=0.0)
    R = A.shape[1]
    part = serving.lora(np.zeros_like(want), np.abs(X.astype(np.float64)), z(A), z(B), index, scale, ranks)
    return np.abs(want) * 2.0 ** -11 + (K + 64) * 2.0 ** -24 * base_abs + (K + R + 8) * 2.0 ** -24 * part + 2.0 ** -24


def _guarded(dev, N, M):
    big = torch.full((N * M + 64,), 0x7E00, dtype=torch.int16, device=dev)
    return big, big[:N * M].view(torch.float16).view(N, M)


SHAPES = [(1, 8, 1, 8), (16, 64, 1, 16), (100, 136, 3, 8), (513, 1000, 8, 24), (300, 4096, 9, 16), (1031, 520, 17, 64),
          (2048, 4096, 32, 40), (700, 4104, 5, 16), (520, 11008, 8, 256), (96, 5000, 32, 8), (4096, 4096, 1, 8),
          (77, 100, 4, 16), (11008, 4096, 8, 16), (8192, 4096, 20, 8)]


@pytest.mark.parametrize("M,K,N,R", SHAPES)
@pytest.mark.parametrize("mixed", [True, False])
def test_f16(M, K, N, R, mixed, dev):
    p = workloads.random_fp16_problem(M + K + N, M, K, N, 0.6)
    rng = np.random.default_rng(M + R)
    n = 1 + N // 2
    ranks = [int(r) for r in rng.integers(0, R + 1, n)] if mixed else None
    A, B, scale = _adapters(rng, n, R, M, K, ranks)
    index = rng.integers(-1 if mixed else 0, n, N).astype(np.int32)
    if mixed and N > 4:
        index[3] = n + 5                        # past the pool: no adapter
    W = bsp.encode(p.W).to_device(dev)
    ad = _dev(dev, A, B, scale, ranks)
    big, Y = _guarded(dev, N, M)
    ws = bsp.new_lora_workspace(W, N, ad, device=dev)
    X = torch.from_numpy(p.X).to(dev)
    idx = torch.from_numpy(index).to(dev)
    bsp.spmm_f16_lora(W, X, ad, idx, Y=Y, workspace=ws)
    first = Y.clone()
    bsp.spmm_f16_lora(W, X, ad, idx, Y=Y, workspace=ws)
    torch.cuda.synchronize()
    assert (big[N * M:] == 0x7E00).all() and not ws[:65536].any()
    assert torch.equal(Y, first)
    W64, X64 = p.W.astype(np.float64), p.X.astype(np.float64)
    z = lambda x: np.where(np.isfinite(x), x, 0).astype(np.float64)
    want = serving.lora(X64 @ W64.T, p.X, z(A), z(B), index, scale, ranks)
    tol = _bound(want, np.abs(X64) @ np.abs(W64).T, p.X, A, B, index, scale, ranks, K)
    worst = np.abs(Y.cpu().numpy() - want) / tol
    assert worst.max() <= 1.0, worst.max()


@pytest.mark.parametrize("M,K,N,R", [(1, 8, 1, 8), (100, 136, 3, 8), (513, 999, 8, 24), (300, 4096, 32, 16),
                                     (1031, 5000, 17, 64), (512, 16384, 8, 16), (12288, 4096, 8, 16)])
def test_w4a4_dequantised(M, K, N, R, dev):
    p = workloads.random_int4_problem(M + K + N, M, K, N)
    rng = np.random.default_rng(M + R)
    A, B, scale = _adapters(rng, 3, R, M, K)
    index = rng.integers(-1, 3, N).astype(np.int32)
    sw, sx = rng.uniform(1e-3, 1e-2, M).astype(np.float32), rng.uniform(0.1, 1, N).astype(np.float32)
    X16 = (p.X * sx[:, None]).astype(np.float16)
    W = bsp.encode(p.W).to_device(dev)
    t = lambda x: torch.from_numpy(x).to(dev)
    big, Y = _guarded(dev, N, M)
    ad = _dev(dev, A, B, scale, None)
    bsp.spmm_w4a4_dq_lora(W, t(bsp.pack_int4(p.X)), t(X16), t(sw), t(sx), ad, t(index), Yh=Y)
    torch.cuda.synchronize()
    assert (big[N * M:] == 0x7E00).all()
    base = (p.X.astype(np.float64) @ p.W.astype(np.float64).T) * sw * sx[:, None].astype(np.float64)
    want = serving.lora(base, X16, A, B, index, scale)
    # the dequantised sum is exact but for its two fp32 products: 2^-22 covers it at any K
    tol = _bound(want, np.abs(base), X16, A, B, index, scale, None, K)
    worst = np.abs(Y.cpu().numpy() - want) / tol
    assert worst.max() <= 1.0, worst.max()


def test_no_adapter_is_the_plain_product(dev):
    p = workloads.random_fp16_problem(3, 300, 512, 6)
    W = bsp.encode(p.W).to_device(dev)
    X = torch.from_numpy(p.X).to(dev)
    A, B, scale = _adapters(np.random.default_rng(0), 2, 8, 300, 512)
    Y = bsp.spmm_f16_lora(W, X, _dev(dev, A, B, scale, None), torch.full((6,), -1, dtype=torch.int32, device=dev))
    assert torch.equal(Y, bsp.spmm_f16(W, X))
    none = bsp.LoraAdapters(torch.empty((0, 8, 512), dtype=torch.float16, device=dev),
                            torch.empty((0, 300, 8), dtype=torch.float16, device=dev))
    Y = bsp.spmm_f16_lora(W, X, none, torch.zeros(6, dtype=torch.int32, device=dev))
    assert torch.equal(Y, bsp.spmm_f16(W, X))


def test_zero_sizes(dev):
    A, B, scale = _adapters(np.random.default_rng(0), 2, 8, 50, 0)
    W = bsp.encode(np.zeros((50, 0), np.float16)).to_device(dev)
    idx = torch.zeros(3, dtype=torch.int32, device=dev)
    Y = bsp.spmm_f16_lora(W, torch.empty((3, 0), dtype=torch.float16, device=dev), _dev(dev, A, B, scale, None), idx)
    assert Y.shape == (3, 50) and not Y.any()
    A, B, scale = _adapters(np.random.default_rng(0), 2, 8, 50, 64)
    W = bsp.encode(np.ones((50, 64), np.float16)).to_device(dev)
    Y = bsp.spmm_f16_lora(W, torch.empty((0, 64), dtype=torch.float16, device=dev), _dev(dev, A, B, scale, None),
                          torch.zeros(0, dtype=torch.int32, device=dev))
    assert Y.shape == (0, 50)


def test_x_off_a_16_byte_boundary(dev):
    p = workloads.random_fp16_problem(5, 200, 256, 4)
    W = bsp.encode(p.W).to_device(dev)
    wide = torch.zeros(4 * 256 + 1, dtype=torch.float16, device=dev)
    wide[1:] = torch.from_numpy(p.X).to(dev).flatten()
    A, B, scale = _adapters(np.random.default_rng(1), 2, 16, 200, 256)
    index = np.array([0, 1, 1, -1], np.int32)
    Y = bsp.spmm_f16_lora(W, wide[1:].view(4, 256), _dev(dev, A, B, scale, None), torch.from_numpy(index).to(dev))
    X64, W64 = p.X.astype(np.float64), p.W.astype(np.float64)
    want = serving.lora(X64 @ W64.T, p.X, A, B, index, scale)
    tol = _bound(want, np.abs(X64) @ np.abs(W64).T, p.X, A, B, index, scale, None, 256)
    assert (np.abs(Y.cpu().numpy() - want) <= tol).all()


def test_graph_replays_and_shared_workspace(dev):
    p = workloads.random_fp16_problem(7, 1000, 4096, 8)
    W = bsp.encode(p.W).to_device(dev)
    X = torch.from_numpy(p.X).to(dev)
    A, B, scale = _adapters(np.random.default_rng(2), 4, 16, 1000, 4096)
    ad, idx = _dev(dev, A, B, scale, None), torch.arange(8, dtype=torch.int32, device=dev) % 5 - 1
    ws = bsp.new_lora_workspace(W, 8, ad, device=dev)
    want, Y = bsp.spmm_f16_lora(W, X, ad, idx, workspace=ws), torch.empty((8, 1000), dtype=torch.float16, device=dev)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            bsp.spmm_f16_lora(W, X, ad, idx, Y=Y, workspace=ws)
    torch.cuda.synchronize()
    for _ in range(3):
        Y.fill_(9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
