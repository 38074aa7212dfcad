"""Heads normed and rotated on the GPU against the oracle, and written to the cache: bit for bit what the
two calls leave there."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import serving, step

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


def _in_order(x, w, eps, positions, freq, rot, inter):
    """The definition in fp32, each operation rounded, the squares added in fours, then neighbours first (heads of 64:
    neighbours first throughout); sines are the nearest floats."""
    y = x.astype(np.float32)
    s = y * y
    if x.shape[-1] > 64:
        s = ((s[..., 0::4] + s[..., 1::4]) + s[..., 2::4]) + s[..., 3::4]
    while s.shape[-1] > 1:
        s = s[..., 0::2] + s[..., 1::2]
    y = y / np.sqrt(s * np.float32(1.0 / x.shape[-1]) + np.float32(eps)) * w.astype(np.float32)
    turns = (positions.astype(np.int64).astype(np.uint64)[:, None] * freq[None, :]).astype(np.int64)
    angle = turns.astype(np.float64) * (2.0 * np.pi / 2.0 ** 64)
    c, z = np.cos(angle).astype(np.float32)[:, None], np.sin(angle).astype(np.float32)[:, None]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    out = y.copy()
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * z, y[..., b] * c + y[..., a] * z
    return out.astype(np.float16)


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 128, False), (128, 64, True), (256, 256, True)])
def test_rounded_in_the_definitions_order(D, rot, inter, dev):
    # A sine is the nearest float but where it lies within 2^-11 of a step from the middle of two (one in 2^10), and a
    # step of one moves a result past an fp16 border once in 2^12: one in 2^21 of the rotated ones. Allowed: 2^-16.
    rng = np.random.default_rng(D + rot)
    n = 1500
    _, Q, K, _ = _fused(rng, n, 9, 2, D, 0, dev)
    positions = rng.integers(-(1 << 17), 1 << 17, n).astype(np.int32)
    w = (1 + 0.3 * rng.normal(0, 1, D)).astype(np.float16)
    freq = bsp.rope_frequencies(rot, device=dev)
    wd = torch.from_numpy(w).to(dev)
    q, k = bsp.qk_norm_rope(Q, K, torch.from_numpy(positions).to(dev), freq, wd, wd, eps=1e-6, interleaved=inter)
    for got, x in ((q, Q), (k, K)):
        want = _in_order(x.cpu().numpy(), w, 1e-6, positions, freq.cpu().numpy().view(np.uint64), rot, inter)
        other = got.cpu().numpy() != want
        assert not other[..., rot:].any() and other.mean() <= 2.0 ** -16, int(other.sum())


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cache_rows_of_any_bits(kind, D, dev):
    # every exponent and the subnormals, rows of one exponent, and rows with an infinity or a NaN in one place. x - o and
    # its quotient are rounded to fp32, by 2^-24 each: a code is the neighbour of the exact quotient's where that lies
    # within 2^-23 of itself of the middle of two (-7.8e-5 + 35040 over 4672, 7.4999999833, is 8).
    rng = np.random.default_rng(D)
    bits = rng.integers(0, 1 << 16, (400, 3, D)).astype(np.uint16)
    bits[bits & 0x7C00 == 0x7C00] ^= 0x4000
    rows = bits.reshape(-1, D)
    rows[::5] = (rows[::5] & 0x83FF) | (rng.integers(0, 31, (rows[::5].shape[0], 1)) << 10)
    x = bits.view(np.float16)
    bad = np.array([[7, 1], [7, 2], [90, 0], [399, 2]])
    for (t, h), v, at in zip(bad, (np.inf, -np.inf, np.nan, np.nan), (0, D - 1, 8, D // 2 + 3)):
        x[t, h, at] = v
    cache = bsp.new_kv_cache(KINDS[kind], 25, 3, 16, D, device=dev)
    X = torch.from_numpy(x).to(dev)
    bsp.kv_append(cache, X, X, torch.arange(400, device=dev))
    flat = lambda t: t.transpose(1, 2).reshape(400, 3, -1).cpu().numpy()
    good = np.ones((400, 3), bool)
    good[bad[:, 0], bad[:, 1]] = False
    codes, words = serving.quantise(np.where(good[..., None], x, 0), kind)
    for c, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c, w = flat(c), flat(w).view(np.uint32)[..., 0]
        assert np.array_equal(w[good], words[good])
        got, want = (np.stack((u & 15, u >> 4), -1).reshape(400, 3, D) if kind == "int4" else u for u in (c, codes))
        off = (got != want) & good[..., None]
        exact = x.astype(np.float64) - np.where(good[..., None], x, 0).min(-1, keepdims=True).astype(np.float64)
        with np.errstate(divide="ignore", invalid="ignore"):
            exact /= (w & 0xFFFF0000).view(np.float32).astype(np.float64)[..., None]
        assert (np.abs(got.astype(int) - want)[off] == 1).all()
        assert (np.abs(exact[off] % 1.0 - 0.5) <= exact[off] * 2.0 ** -23).all()
        assert not c[~good].any() and (w[~good] == 0x7FC07E00).all()
