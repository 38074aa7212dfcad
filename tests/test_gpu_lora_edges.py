"""Adapters beside a projection at their edges: sums that pass the fp16 and the
fp32 range, per-adapter ranks, indices past the pool and unaligned activations
through both entry points."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
import workloads
from oracle import serving
from test_gpu_lora import _adapters, _bound, _dev, _guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


SHAPES = [(70, 64, 1), (520, 1024, 8), (300, 1000, 20), (300, 4096, 32), (700, 11008, 8), (5, 100, 2)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("R", [8, 16, 24, 40, 64])
@pytest.mark.parametrize("kind", ["f16", "w4a4"])
def test_sums_past_the_fp32_range(M, K, N, R, kind, dev):
    # t_n is infinite at every rank position in use and B has one sign per output:
    # an infinity of that sign, whatever the loads past the rank hold
    rng = np.random.default_rng(M + R)
    ranks = [R, max(1, R - 7), 1]
    A = np.abs(rng.normal(1, 0.1, (3, R, K))).astype(np.float16)
    B = (np.abs(rng.normal(1, 0.1, (3, M, R))) * np.where(np.arange(M) % 3, 1, -1)[None, :, None]).astype(np.float16)
    for a, r in enumerate(ranks):
        A[a, r:], B[a, :, r:] = np.nan, np.nan
    ad = _dev(dev, A, B, np.full(3, 3e38, np.float32), ranks)
    index = (np.arange(N) % 4 - (N > 1)).astype(np.int32)      # -1 and past the pool: no adapter
    idx = torch.from_numpy(index).to(dev)
    t = lambda x: torch.from_numpy(x).to(dev)
    if kind == "f16":
        p = workloads.random_fp16_problem(M + K, M, K, N, 0.5)
        X = np.abs(p.X) + np.float16(1)
        W = bsp.encode(p.W).to_device(dev)
        Y = bsp.spmm_f16_lora(W, t(X), ad, idx)
        plain = bsp.spmm_f16(W, t(X))
    else:
        p = workloads.random_int4_problem(M + K, M, K, N)
        W, X = bsp.encode(p.W).to_device(dev), t(bsp.pack_int4(p.X))
        sw, sx = t(np.full(M, 1e-3, np.float32)), t(np.ones(N, np.float32))
        Y = bsp.spmm_w4a4_dq_lora(W, X, t(np.ones((N, K), np.float16)), sw, sx, ad, idx)
        plain = t((p.X.astype(np.float64) @ p.W.astype(np.float64).T * np.float32(1e-3)).astype(np.float16))
    torch.cuda.synchronize()
    want = np.where(np.arange(M) % 3, np.inf, -np.inf)
    for n, a in enumerate(index):
        if 0 <= a < 3:
            assert np.array_equal(Y[n].cpu().numpy(), want), (n, a)
        else:
            assert (Y[n].float() - plain[n].float()).abs().max() <= 2.0 ** -10 * plain[n].float().abs().max() + 2.0 ** -24
