"""Heads normed and rotated on the GPU against the oracle, and written to the cache: bit for bit what the
two calls leave there."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
KINDS = {"fp16": bsp.FP16, "int8": bsp.INT8, "int4": bsp.INT4}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _angles(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))


def _close(got, x, weight, eps, positions, rot, inter):
    """The sum of squares: a lane's chain of 8 fma and up to 5 additions, halved by the root, then at most 5 roundings:
    under 2^-20 of a value; sine and cosine 2^-21 off; two products and a sum: under 2^-19 of |y1| + |y2| in all, and
    half a step of fp16."""
    y = step.normed(x, weight, eps)
    want, size = step.rotated(y, positions, _angles(rot), inter) if rot else (y, np.abs(y))
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    fine = np.abs(want) < 65000
    assert (err <= np.abs(want) * 2.0 ** -11 + size * 2.0 ** -19 + 2.0 ** -25)[fine].all(), err.max()


def _fused(rng, n, hq, hkv, D, pad, dev):
    """A fused projection's rows (`pad` elements behind them), and its query, key and value slices."""
    x = rng.normal(0, 1, (n, (hq + 2 * hkv) * D + pad)) * np.exp(rng.normal(0, 1, (n, 1)))
    wide = torch.from_numpy(x.astype(np.float16)).to(dev)
    cut = lambda a, h: wide[:, a * D:(a + h) * D].unflatten(1, (h, D))
    return wide, cut(0, hq), cut(hq, hkv), cut(hq + hkv, hkv)


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 32), (128, 96), (128, 0), (256, 256),
                                   (256, 48)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", ["both", "none", "q"])
@pytest.mark.parametrize("n,hq,hkv,pad", [(1, 1, 1, 0), (3, 5, 2, 0), (2, 9, 3, 1), (5, 32, 32, 8)])
def test_norm_and_rotation(D, rot, inter, norm, n, hq, hkv, pad, dev):
    rng = np.random.default_rng(D + rot * 3 + n + inter)
    _, Q, K, _ = _fused(rng, n, hq, hkv, D, pad, dev)
    positions = rng.integers(0, 1 << 20, n).astype(np.int32)
    positions[0] = (1 << 31) - 1 if n > 1 else 0
    w = [torch.from_numpy((1 + 0.3 * rng.normal(0, 1, D)).astype(np.float16)).to(dev) for _ in range(2)]
    wq, wk = (w[0] if norm != "none" else None), (w[1] if norm == "both" else None)
    freq = bsp.rope_frequencies(rot, device=dev) if rot else None
    q, k = bsp.qk_norm_rope(Q, K, torch.from_numpy(positions).to(dev), freq, wq, wk, eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    for got, x, ww in ((q, Q, wq), (k, K, wk)):
        _close(got, x.cpu().numpy(), None if ww is None else ww.cpu().numpy(), 1e-5, positions, rot, inter)


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 128, False), (128, 64, True), (256, 128, False)])
@pytest.mark.parametrize("n,hq,hkv,pad,page", [(1, 4, 4, 0, 16), (7, 10, 2, 0, 16), (33, 3, 5, 1, 32), (130, 8, 1, 8, 64)])
def test_written_to_the_cache(kind, D, rot, inter, n, hq, hkv, pad, page, dev):
    rng = np.random.default_rng(n + D + rot)
    _, Q, K, V = _fused(rng, n, hq, hkv, D, pad, dev)
    pages = -(-n // page) + 2
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[n // 2] = [-1, pages * page, 1 << 40][n % 3]        # outside the cache: skipped
    slots = torch.from_numpy(slots).to(dev)
    positions = torch.from_numpy(rng.integers(0, 100000, n).astype(np.int32)).to(dev)
    w = torch.from_numpy((1 + 0.3 * rng.normal(0, 1, D)).astype(np.float16)).to(dev)
    freq = bsp.rope_frequencies(rot, device=dev)
    args = dict(q_weight=w, k_weight=w, eps=1e-6, interleaved=inter)
    one, two = (bsp.new_kv_cache(KINDS[kind], pages, hkv, page, D, device=dev) for _ in range(2))
    q = bsp.qk_norm_rope_append(Q, K, V, positions, freq, one, slots, **args)
    q2, k2 = bsp.qk_norm_rope(Q, K, positions, freq, **args)
    bsp.kv_append(two, k2, V, slots)
    torch.cuda.synchronize()
    assert torch.equal(q, q2)
    for name in ("k", "v", "k_scale", "v_scale"):
        a, b = getattr(one, name), getattr(two, name)
        assert (a is None and b is None) or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_in_place_and_beside_it(dev):
    rng = np.random.default_rng(2)
    wide, Q, K, V = _fused(rng, 19, 6, 2, 128, 8, dev)
    positions = torch.arange(19, dtype=torch.int32, device=dev)
    freq = bsp.rope_frequencies(128, device=dev)
    q, k = bsp.qk_norm_rope(Q, K, positions, freq)
    before = wide.clone()
    bsp.qk_norm_rope(Q, K, positions, freq, Qo=Q, Ko=K)
    torch.cuda.synchronize()
    assert torch.equal(Q, q) and torch.equal(K, k)
    assert torch.equal(wide[:, 8 * 128:], before[:, 8 * 128:])


def test_positions_are_exact_far_out(dev):
    # pair i at position p and at position 0 turned by hand: far positions lose nothing; negative ones turn back
    D = 64
    x = torch.randn(1, 1, D, device=dev).half().expand(7, 1, D).contiguous()
    p = np.array([0, 1, -1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31], np.int64)
    pos = torch.from_numpy(p.astype(np.int32)).to(dev)
    q, _ = bsp.qk_norm_rope(x, x, pos, bsp.rope_frequencies(D, 500000.0, device=dev))
    y = x.cpu().numpy().astype(np.float64)
    want, size = step.rotated(y, p, _angles(D, 500000.0), False)
    assert (np.abs(q.cpu().numpy() - want) <= np.abs(want) * 2.0 ** -11 + size * 2.0 ** -19 + 2.0 ** -25).all()
    # whole turns: an angle of exactly a quarter turn per position
    quarter = bsp.rope_frequencies(D, angles=np.full(D // 2, np.pi / 2), device=dev)
    q, _ = bsp.qk_norm_rope(x, x, torch.tensor([0, 4, 8, 1 << 30, 1, 2, 3], dtype=torch.int32, device=dev), quarter)
    assert torch.equal(q[:4], x[:4])
    a, b = x[0, 0, :32], x[0, 0, 32:]
    assert torch.equal(q[4, 0], torch.cat((-b, a))) and torch.equal(q[5, 0], -x[0, 0])


def test_rows_that_are_not_finite_stay_alone(dev):
    x = torch.randn(3, 4, 128, device=dev).half()
    x[1, 2, 5] = float("nan")
    x[2, 0, 7] = float("inf")
    pos = torch.arange(3, dtype=torch.int32, device=dev)
    w = torch.ones(128, dtype=torch.float16, device=dev)
    q, _ = bsp.qk_norm_rope(x, x, pos, bsp.rope_frequencies(128, device=dev), q_weight=w)
    bad = ~torch.isfinite(q).all(-1)
    assert bad.nonzero().tolist() == [[1, 2], [2, 0]]
    cache = bsp.new_kv_cache(bsp.INT8, 1, 4, 16, 128, device=dev)
    bsp.qk_norm_rope_append(x, x, x, pos, None, cache, torch.arange(3, device=dev))
    k, v = bsp.kv_gather(cache, torch.arange(3, device=dev))
    assert torch.isnan(k).all(-1).nonzero().tolist() == [[1, 2], [2, 0]] and torch.equal(k.isnan(), v.isnan())


def test_streams_graph_and_empty_calls(dev):
    g = torch.Generator(device=dev).manual_seed(5)
    Q, K, V = (torch.randn(40, h, 128, generator=g, device=dev).half() for h in (8, 2, 2))
    pos = torch.arange(40, dtype=torch.int32, device=dev)
    freq = bsp.rope_frequencies(128, device=dev)
    slots = torch.arange(40, device=dev)
    caches = [bsp.new_kv_cache(bsp.INT4, 4, 2, 16, 128, device=dev) for _ in range(3)]
    ref = bsp.qk_norm_rope_append(Q, K, V, pos, freq, caches[0], slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = bsp.qk_norm_rope_append(Q, K, V, pos, freq, caches[1], slots, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(q, ref) and torch.equal(caches[0].k, caches[1].k)
    out = torch.empty_like(Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsp.qk_norm_rope_append(Q, K, V, pos, freq, caches[2], slots, Qo=out)
    for k in range(3):
        Q.copy_(torch.randn(Q.shape, generator=g, device=dev).half())
        pos += 1000
        graph.replay()
        ref = bsp.qk_norm_rope_append(Q, K, V, pos, freq, caches[0], slots)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(caches[0].k, caches[2].k)
    none = torch.empty(0, 8, 128, dtype=torch.float16, device=dev)
    empty = torch.empty(0, dtype=torch.int32, device=dev)
    q, k = bsp.qk_norm_rope(none, none[:, :2], empty, freq)
    assert q.shape == (0, 8, 128) and k.shape == (0, 2, 128)


def test_many_tokens(dev):
    rng = np.random.default_rng(8)
    n = 3001
    _, Q, K, V = _fused(rng, n, 16, 4, 128, 0, dev)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    w = torch.from_numpy((1 + 0.3 * rng.normal(0, 1, 128)).astype(np.float16)).to(dev)
    freq = bsp.rope_frequencies(128, device=dev)
    cache = bsp.new_kv_cache(bsp.INT8, 200, 4, 16, 128, device=dev)
    q = bsp.qk_norm_rope_append(Q, K, V, pos, freq, cache, pos.long() + 100, w, w, eps=1e-5)
    q1, k1 = bsp.qk_norm_rope(Q[2900:2930], K[2900:2930], pos[2900:2930], freq, w, w, eps=1e-5)
    assert torch.equal(q[2900:2930], q1)      # the same token in a short call: the same bits
    k, v = bsp.kv_gather(cache, pos.long() + 100)
    two = bsp.new_kv_cache(bsp.INT8, 200, 4, 16, 128, device=dev)
    bsp.kv_append(two, k1, V[2900:2930], pos.long()[:30])
    k2, v2 = bsp.kv_gather(two, pos.long()[:30])
    assert torch.equal(k[2900:2930], k2) and torch.equal(v[2900:2930], v2)
    _close(q[:40], Q[:40].cpu().numpy(), w.cpu().numpy(), 1e-5, np.arange(40), 128, False)
