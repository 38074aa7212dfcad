"""The decode-step operators over more of what they accept: long runs of tiles
per wavefront, more sequences than a wavefront has lanes, pages and groups of
other sizes, more heads than the workspace counts, adapters on int4 weights with
ranks and indices of all kinds, and one workspace for calls of every operator."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
import workloads
from oracle import serving
from test_gpu_attention_tree import Case
from test_gpu_lora import _adapters, _bound, _dev, _guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
KINDS = ["fp16", "int8", "int4"]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,n", [(1, 4200), (1, 8500), (64, 1100), (64, 2200), (20, 3000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_more_than_32_tiles_per_wavefront(kind, T, n, D, dev):
    # pages are looked up 32 tiles at a time: one workgroup walks all of these
    c = Case(n + T, [(T, n)], 2, 1, D, kind, 16, dev)
    c.check(c.run(split=False))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [64, 65, 130])
@pytest.mark.parametrize("T,hq", [(1, 4), (5, 8)])
@pytest.mark.parametrize("split", [True, False])
def test_more_sequences_than_lanes(kind, B, T, hq, split, dev):
    # lengths from 0 on; empty sequences and ones without queries about the edges of 64
    rng = np.random.default_rng(B + T)
    lens = []
    for b in range(B):
        n = int(rng.integers(T, 120)) if b % 9 else int(rng.integers(300, 900))
        lens.append((0, n) if b in (0, 62, 64, 127) else (0, 0) if b in (1, 63, 128) else (T, T) if b in (65, 129) else
                    (int(rng.integers(1, T + 1)), n))
    c = Case(B * 3 + T, lens, hq, 2, 64, kind, 16, dev)
    c.check(c.run(split=split))


@pytest.mark.parametrize("kind", KINDS)
def test_long_sequences_past_the_first_64(kind, dev):
    # what is split, and joined by a kernel of its own, lies in the second and third 64
    lens = [(1, 3)] * 70 + [(6, 4000), (0, 0)] + [(1, 17)] * 60 + [(3, 2500)]
    c = Case(133, lens, 16, 2, 64, kind, 32, dev)
    c.check(c.run())


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("kind", KINDS)
def test_more_heads_than_the_workspace_counts(kind, split, dev):
    # 4 x 4100 arrivals do not fit 64 KiB of counters: no split, with a workspace or without
    c = Case(9, [(1, 20), (2, 33), (1, 1), (1, 40)], 4100, 4100, 64, kind, 16, dev)
    n = bsp.attention_workspace_bytes(c.cache, 4, 2, 4100, 3)
    assert n == 0
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev) if split else None
    c.check(c.run(split=split, ws=ws))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [256, 1024, 4096])
def test_large_pages(kind, page, dev):
    c = Case(page, [(3, 5000), (1, page), (2, page + 1), (1, 7)], 4, 2, 128, kind, page, dev)
    c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,T,D", [(40, 4, 64), (130, 1, 128), (33, 7, 128), (300, 2, 64), (70, 1, 256)])
def test_wide_groups(kind, group, T, D, dev):
    c = Case(group + T, [(T, 333), (1, 1500)], 2 * group, 2, D, kind, 16, dev)
    c.check(c.run())


W4A4 = [(100, 136, 3, 8), (513, 999, 8, 24), (300, 4096, 32, 64), (1031, 5000, 17, 40), (512, 16384, 8, 16),
        (5000, 2048, 8, 256), (16384, 2048, 8, 16), (64, 20000, 4, 32), (7, 4096, 1, 8)]


@pytest.mark.parametrize("M,K,N,R", W4A4)
@pytest.mark.parametrize("off", [0, 1])
def test_w4a4_ranks_indices_and_alignment(M, K, N, R, off, dev):
    p = workloads.random_int4_problem(M + K + N, M, K, N)
    rng = np.random.default_rng(M + R)
    n = 2 + N // 2
    ranks = [int(r) for r in rng.integers(-1, R + 3, n)]                  # clamped to 0 .. R
    A, B, scale = _adapters(rng, n, R, M, K, [min(max(r, 0), R) for r in ranks])
    index = rng.integers(-1, n + 1, N).astype(np.int32)
    index[N // 2] = 2 ** 31 - 1 if N > 2 else 0
    sw, sx = rng.uniform(1e-3, 1e-2, M).astype(np.float32), rng.uniform(0.1, 1, N).astype(np.float32)
    X16 = (p.X * sx[:, None]).astype(np.float16)
    W, Xp = bsp.encode(p.W).to_device(dev), bsp.pack_int4(p.X)

    def t(x, off=0):
        flat = torch.zeros(x.size + off, dtype=torch.from_numpy(x[:0]).dtype, device=dev)
        flat[off:] = torch.from_numpy(x).to(dev).flatten()
        return flat[off:].view(x.shape)

    big, Y = _guarded(dev, N, M)
    ad = _dev(dev, A, B, scale, ranks)
    ws = bsp.new_lora_workspace(W, N, ad, device=dev)
    bsp.spmm_w4a4_dq_lora(W, t(Xp, off), t(X16, off), t(sw), t(sx), ad, t(index), Yh=Y, workspace=ws)
    torch.cuda.synchronize()
    assert (big[N * M:] == 0x7E00).all() and not ws[:65536].any()
    base = (p.X.astype(np.float64) @ p.W.astype(np.float64).T) * sw * sx[:, None].astype(np.float64)
    z = lambda x: np.where(np.isfinite(x), x, 0).astype(np.float64)
    want = serving.lora(base, X16, z(A), z(B), index, scale, ranks)
    tol = _bound(want, np.abs(base), X16, A, B, index, scale, ranks, K)
    worst = np.abs(Y.cpu().numpy() - want) / tol
    assert worst.max() <= 1.0, worst.max()


def test_one_workspace_for_calls_of_every_operator(dev):
    t = lambda x: torch.from_numpy(x).to(dev)
    rng = np.random.default_rng(0)
    f = workloads.random_fp16_problem(1, 700, 11008, 8, 0.4)              # splits K
    q = workloads.random_int4_problem(2, 300, 16384, 8)
    Wf, Wq = bsp.encode(f.W).to_device(dev), bsp.encode(q.W).to_device(dev)
    af, aq = (_dev(dev, *_adapters(rng, 3, 16, M, K), None) for M, K in ((700, 11008), (300, 16384)))
    idx = t(np.array([0, 1, 2, -1, 0, 1, 2, 2], np.int32))
    Xf, Xq, Xq16 = t(f.X), t(bsp.pack_int4(q.X)), t(q.X.astype(np.float16))
    sw, sx = t(np.full(300, 1e-3, np.float32)), t(np.full(8, 0.5, np.float32))
    one = Case(3, [(1, 5000), (1, 300)], 8, 2, 128, "int8", 16, dev)         # joined by its last chunk
    tree = Case(4, [(12, 3000)], 16, 2, 64, "fp16", 32, dev)                 # by a kernel of its own
    calls = [lambda ws: bsp.spmm_f16_lora(Wf, Xf, af, idx, workspace=ws), lambda ws: one.run(ws=ws),
             lambda ws: bsp.spmm_w4a4_dq_lora(Wq, Xq, Xq16, sw, sx, aq, idx, workspace=ws),
             lambda ws: bsp.spmm_f16(Wf, Xf, workspace=ws), lambda ws: tree.run(ws=ws),
             lambda ws: bsp.spmm_w4a4(Wq, Xq, 8, workspace=ws)]
    new = lambda: torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    want = [call(new()) for call in calls]
    one.check(want[1]), tree.check(want[4])
    ws = new()
    for order in ([0, 1, 2, 3, 4, 5], [5, 1, 0, 4, 2, 3], [4, 0, 1, 3, 1, 2, 5, 0]):
        got = [(i, calls[i](ws)) for i in order]
        torch.cuda.synchronize()
        for i, y in got:
            assert torch.equal(y, want[i]), i
        assert not ws[:65536].any()
