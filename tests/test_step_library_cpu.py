"""Refusals, on the host, of the operators from the hidden states to the cache: every call here fails (or
launches nothing) before any HIP call, the pointers are never dereferenced."""
import ctypes
import math

import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step
from test_serving_library_cpu import BAD_CACHES, cache

FAKE = 0x1000
INT32_MAX = 2 ** 31 - 1


def test_pages():
    L = bsp.load_library()
    base = dict(sequences=3, table_width=4, page_size=16, pool=8, block_table=FAKE, lens=FAKE, held=FAKE, free_pages=FAKE)

    def call(none=False, keep=FAKE, new=FAKE, mask=None, rows=8, slots=FAKE, positions=FAKE, sequences_=FAKE,
             q_start=FAKE, kv_lens=FAKE, **kw):
        d = bsp._KVPagesDesc(*(dict(base, **kw)[n] for n, _ in bsp._KVPagesDesc._fields_))
        return L.kv_pages_step(None if none else ctypes.byref(d), keep, new, mask, rows, slots, positions, sequences_,
                               q_start, kv_lens, None)

    for bad in (dict(none=True), dict(sequences=-1), dict(table_width=-1), dict(pool=-1), dict(rows=-1),
                dict(page_size=8), dict(page_size=48), dict(page_size=8192), dict(block_table=None), dict(lens=None),
                dict(held=None), dict(free_pages=None), dict(new=None), dict(slots=None), dict(positions=None),
                dict(sequences_=None), dict(q_start=None), dict(kv_lens=None), dict(keep=FAKE + 2), dict(slots=FAKE + 4),
                dict(mask=FAKE + 4), dict(lens=FAKE + 1), dict(free_pages=FAKE + 2)):
        assert call(**bad) == bsp.E_ARG, bad
    assert call(sequences=bsp.PAGES_MAX_SEQUENCES + 1) == bsp.E_UNSUPPORTED
    for bad in (dict(rows=1 << 28), dict(table_width=1 << 27), dict(pool=1 << 32), dict(pool=INT32_MAX - 11),
                dict(sequences=4096, table_width=1 << 19), dict(table_width=(INT32_MAX - 4095) // 16)):
        assert call(**bad) == bsp.E_OVERFLOW, bad


def _rotation(**kw):
    a = dict(dict(rot=64, interleaved=0, freq=FAKE, positions=FAKE, q_weight=None, k_weight=None, eps=1e-6), **kw)
    return bsp._ROTATION.pack(*(a[n] or 0 for n in ("rot", "interleaved", "freq", "positions", "q_weight", "k_weight", "eps")))


def test_heads():
    L = bsp.load_library()

    def call(none=False, Q=FAKE, qs=512, K=FAKE, ks=128, n=4, hq=8, hkv=2, D=64, Qo=FAKE, qos=512, Ko=FAKE, kos=128, **kw):
        r = None if none else _rotation(**kw)
        return L.qk_norm_rope_f16(Q, qs, K, ks, n, hq, hkv, D, r, Qo, qos, Ko, kos, None)

    for bad in (dict(none=True), dict(n=-1), dict(hq=-1), dict(hkv=-1), dict(Q=None), dict(K=None), dict(Qo=None),
                dict(Ko=None), dict(qs=511), dict(ks=127), dict(qos=0), dict(kos=127), dict(Q=FAKE + 1), dict(Ko=FAKE + 1),
                dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(q_weight=FAKE + 2), dict(k_weight=FAKE + 8),
                dict(freq=None), dict(positions=None), dict(freq=FAKE + 4), dict(positions=FAKE + 2)):
        assert call(**bad) == bsp.E_ARG, bad
    for bad in (dict(D=96), dict(D=0), dict(rot=80), dict(rot=-16), dict(rot=8), dict(rot=20)):
        assert call(**bad) == bsp.E_UNSUPPORTED, bad
    assert call(n=1 << 28) == bsp.E_OVERFLOW and call(n=1 << 25, hq=8, hkv=2) == bsp.E_OVERFLOW
    assert call(hq=1 << 30, qs=1 << 40, qos=1 << 40) == bsp.E_OVERFLOW
    assert call(n=0, Q=None, K=None) == bsp.OK and call(hq=0, hkv=0, Q=None) == bsp.OK


def test_heads_to_the_cache():
    L = bsp.load_library()

    def call(c=cache(), Q=FAKE, V=FAKE, vs=128, n=4, hq=8, slots=FAKE, none=False, **kw):
        r = None if none else _rotation(**kw)
        return L.qk_norm_rope_append_f16(Q, 512, FAKE, 128, V, vs, n, hq, r, None if c is None else ctypes.byref(c), slots,
                                         FAKE, 512, None)

    for bad, status in BAD_CACHES:
        assert call(c=cache(**bad)) == status, bad
    for bad in (dict(c=None), dict(none=True), dict(V=None), dict(vs=127), dict(slots=None), dict(slots=FAKE + 4), dict(n=-1),
                dict(hq=-1), dict(Q=None), dict(eps=-1.0)):
        assert call(**bad) == bsp.E_ARG, bad
    assert call(rot=128) == bsp.E_UNSUPPORTED and call(n=1 << 28) == bsp.E_OVERFLOW
    assert call(n=0, Q=None, V=None, slots=None) == bsp.OK


def _tokens(**kw):
    a = dict(dict(n=3, K=64, X=FAKE, x_stride=64, residual=None, residual_stride=0, weight=None, eps=1e-6, hidden=None,
                  hidden_stride=0, x16=None, x16_stride=0, scale=FAKE), **kw)
    return bsp._TOKENS.pack(*(v or 0 for v in a.values()))


def test_tokens():
    L = bsp.load_library()

    def call(none=False, dtype=bsp.INT8, codes=FAKE, stride=64, **kw):
        return L.quantize_tokens_f16(None if none else _tokens(**kw), dtype, codes, stride, None)

    pair = dict(residual=FAKE, hidden=FAKE, residual_stride=64, hidden_stride=64)
    for bad in (dict(none=True), dict(dtype=bsp.FP16), dict(dtype=bsp.INT2), dict(dtype=9), dict(n=-1), dict(K=-1),
                dict(X=None), dict(codes=None), dict(scale=None), dict(stride=63), dict(dtype=bsp.INT4, stride=31),
                dict(x_stride=63), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(residual=FAKE),
                dict(hidden=FAKE), dict(pair, residual_stride=63), dict(pair, hidden_stride=1), dict(x16=FAKE, x16_stride=2),
                dict(X=FAKE + 1), dict(scale=FAKE + 2), dict(weight=FAKE + 1)):
        assert call(**bad) == bsp.E_ARG, bad
    for bad in (dict(K=1 << 25), dict(n=1 << 31), dict(n=1 << 30, K=1 << 12)):
        assert call(**bad) == bsp.E_OVERFLOW, bad
    assert call(n=0, X=None) == bsp.OK and call(K=0, X=None) == bsp.OK

    def back(codes=FAKE, stride=64, dtype=bsp.INT8, scale=FAKE, n=3, K=64, X=FAKE, xs=64):
        return L.dequantize_tokens_f16(codes, stride, dtype, scale, n, K, X, xs, None)

    for bad in (dict(codes=None), dict(stride=63), dict(dtype=bsp.FP16), dict(scale=None), dict(n=-1), dict(K=-1),
                dict(X=None), dict(xs=63), dict(X=FAKE + 1), dict(scale=FAKE + 1)):
        assert back(**bad) == bsp.E_ARG, bad
    assert back(n=1 << 31) == bsp.E_OVERFLOW and back(n=0, X=None) == bsp.OK


def test_product():
    L = bsp.load_library()

    def call(tiles=FAKE, M=64, K=128, X=FAKE, xs=128, N=4, sw=FAKE, sx=FAKE, Y=FAKE, ys=64, ws=None, wb=0):
        return L.gemm_w8a8_dq(tiles, M, K, X, xs, N, sw, sx, Y, ys, ws, wb, None)

    for bad in (dict(M=-1), dict(K=-1), dict(N=-1), dict(tiles=None), dict(X=None), dict(sw=None), dict(sx=None),
                dict(Y=None), dict(ys=63), dict(xs=127), dict(xs=136), dict(xs=112), dict(X=FAKE + 8), dict(tiles=FAKE + 4),
                dict(Y=FAKE + 1), dict(sw=FAKE + 2), dict(sx=FAKE + 2), dict(wb=-1), dict(wb=256),
                dict(ws=FAKE + 16, wb=1 << 20)):
        assert call(**bad) == bsp.E_ARG, bad
    for bad in (dict(K=131072, xs=131072), dict(M=1 << 31, ys=1 << 32), dict(N=1 << 31)):
        assert call(**bad) == bsp.E_OVERFLOW, bad
    assert call(M=0, Y=None) == bsp.OK and call(N=0, X=None) == bsp.OK
    n = ctypes.c_int64(-1)
    assert L.gemm_w8a8_workspace_bytes(64, 64, 1, None) == bsp.E_ARG
    assert L.gemm_w8a8_workspace_bytes(-1, 64, 1, ctypes.byref(n)) == bsp.E_ARG
    assert L.gemm_w8a8_workspace_bytes(64, 131072, 1, ctypes.byref(n)) == bsp.E_OVERFLOW
    for M, K, N in ((0, 64, 4), (64, 0, 4), (64, 64, 0)):
        assert bsp.gemm_workspace_bytes(M, K, N) == 0


def test_workspace_of_the_product_is_checked():
    L = bsp.load_library()
    for M, K, N in ((4096, 4096, 1), (1024, 11008, 33), (512, 11008, 140), (64, 131071, 300)):
        need = bsp.gemm_workspace_bytes(M, K, N)
        assert 0 <= need < 1 << 30
        if need:
            xs = -(-K // 16) * 16
            assert L.gemm_w8a8_dq(FAKE, M, K, FAKE, xs, N, FAKE, FAKE, FAKE, M, FAKE, need - 1, None) == bsp.E_CAPACITY


def test_sizes_past_what_the_kernels_index():
    L = bsp.load_library()

    def product(M, K, xs, N, ys):
        return L.gemm_w8a8_dq(FAKE, M, K, FAKE, xs, N, FAKE, FAKE, FAKE, ys, None, 0, None)

    assert product(16, 64, 1 << 23, 4, 16) == bsp.E_OVERFLOW                       # rows too far apart
    assert product((1 << 26) - 127, 64, 64, 4, 1 << 26) == bsp.E_OVERFLOW          # more rows than a launch has tiles
    n = ctypes.c_int64(0)
    assert L.gemm_w8a8_workspace_bytes((1 << 26) - 127, 64, 4, ctypes.byref(n)) == bsp.E_OVERFLOW
    assert L.gemm_w8a8_workspace_bytes((1 << 26) - 128, 64, 4, ctypes.byref(n)) == bsp.OK

    def heads(hq, hkv):
        return L.qk_norm_rope_f16(FAKE, hq * 64, FAKE, hkv * 64, 1, hq, hkv, 64, _rotation(), FAKE, hq * 64, FAKE, hkv * 64, None)

    assert heads((1 << 20) + 1, 1) == bsp.E_OVERFLOW and heads(1, (1 << 20) + 1) == bsp.E_OVERFLOW


@pytest.mark.parametrize("M,K", [(4096, 11008), (1024, 11008), (64, 131071), (33, 40000), (16, 4096)])
def test_more_tokens_need_no_less_workspace(M, K):
    sizes = [bsp.gemm_workspace_bytes(M, K, N) for N in list(range(1, 40)) + list(range(41, 5000, 37)) + [1 << 30]]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("M,K", [(1, 1), (16, 64), (17, 65), (5, 200), (40, 16), (33, 1000)])
def test_laid_out_weights(M, K):
    rng = np.random.default_rng(M + K)
    W = rng.integers(-128, 128, (M, K)).astype(np.int8)
    enc = bsp.encode_int8(W, np.ones(M, np.float32))
    bands, ktiles = -(-M // 16), -(-K // 64)
    assert enc.tiles.shape == (bands * ktiles * 1024,)
    t = enc.tiles.view(np.int8).reshape(bands, ktiles, 4, 16, 16)      # band, tile, piece of columns, row, column
    full = t.transpose(0, 3, 1, 2, 4).reshape(bands * 16, ktiles * 64)
    assert np.array_equal(full[:M, :K], W) and not full[M:].any() and not full[:, K:].any()
    strided = np.zeros((M, K + 3), np.int8)
    strided[:, :K] = W
    L = bsp.load_library()
    out = np.empty_like(enc.tiles)
    assert L.encode_int8_tiles(bsp._np_ptr(strided), M, K, K + 3, bsp._np_ptr(out)) == bsp.OK
    assert np.array_equal(out, enc.tiles)


def test_laying_out_refuses():
    L = bsp.load_library()
    assert L.int8_tiles_bytes(-1, 4) == -1 and L.int8_tiles_bytes(17, 65) == 4096 and L.int8_tiles_bytes(0, 65) == 0
    a = np.zeros(4096, np.uint8)
    p = bsp._np_ptr(a)
    for bad in ((None, 1, 1, 1, p), (p, 1, 1, 1, None), (p, -1, 1, 1, p), (p, 1, -1, 1, p), (p, 1, 4, 3, p)):
        assert L.encode_int8_tiles(*bad) == bsp.E_ARG, bad
    assert L.encode_int8_tiles(p, 1, 131072, 131072, p) == bsp.E_OVERFLOW
    assert L.encode_int8_tiles(None, 0, 5, 5, None) == bsp.OK
    assert L.int8_tiles_bytes(1, 131072) == -1 and L.int8_tiles_bytes(1 << 62, 64) == -1
    with pytest.raises(bsp.BspError):
        bsp.encode_int8(np.zeros((1, 131072), np.int8), np.ones(1))
    with pytest.raises(TypeError):
        bsp.encode_int8(np.zeros((2, 2), np.float32), np.ones(2))
    with pytest.raises(ValueError):
        bsp.encode_int8(np.zeros((2, 2), np.int8), np.ones(3))


def test_frequencies():
    torch = pytest.importorskip("torch")
    f = bsp.rope_frequencies(128, 10000.0, device="cpu").numpy().view(np.uint64)
    want = 10000.0 ** (-2.0 * np.arange(64) / 128) / (2 * np.pi)
    assert np.abs(f.astype(np.float64) / 2.0 ** 64 - want).max() < 2.0 ** -53
    # a whole number of turns and negative angles
    f = bsp.rope_frequencies(4, angles=[2 * np.pi, -np.pi], device="cpu")
    assert f.tolist() == [0, -2 ** 63]
    assert bsp.rope_frequencies(0, device="cpu").shape == (0,)
    for bad in (dict(rot=4, angles=[1.0]), dict(rot=4, angles=[1.0, np.nan]), dict(rot=2, angles=[np.inf])):
        with pytest.raises(ValueError):
            bsp.rope_frequencies(**bad, device="cpu")
    assert isinstance(bsp.rope_frequencies(16, device="cpu"), torch.Tensor)


def test_python_refuses_what_is_not_on_the_device():
    torch = pytest.importorskip("torch")
    i32, f16 = torch.int32, torch.float16
    t = torch.zeros(4, dtype=i32)
    with pytest.raises(TypeError):
        bsp.KVPages(torch.zeros(2, 2, dtype=i32), t[:2], t[:2], t, 16)
    with pytest.raises(ValueError):
        bsp.KVPages(t, t, t, t, 16)
    x = torch.zeros(2, 64, dtype=f16)
    with pytest.raises(ValueError):
        bsp.quantize_tokens(x, bsp.INT8)
    h = torch.zeros(2, 4, 64, dtype=f16)
    with pytest.raises(ValueError):
        bsp.qk_norm_rope(h, h, t[:2], None)
    with pytest.raises((TypeError, ValueError)):
        bsp.dequantize_tokens(torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2), bsp.INT8, 64)
    with pytest.raises(TypeError):
        bsp.DenseInt8(16, 64, torch.zeros(1024, dtype=torch.uint8), torch.zeros(16))


# ---- the oracle itself, against plain instances of the definitions ----

def test_oracle_pages():
    s = step.Pages([[3, 9, 9], [5, 6, 9]], [16, 20], [1, 2], [7, 8], 16)
    out = s.step([16, 3], [17, 1], 20)
    assert out[0] == [6 * 16 + i for i in range(16)] + [8 * 16] + [5 * 16 + 3, -1, -1]      # page 6 first, it was given back
    assert out[1] == list(range(16, 33)) + [3, 0, 0] and out[2] == [0] * 17 + [1, -1, -1]
    assert out[3] == [0, 17, 18] and out[4] == [33, 4] and s.free == [7] and s.held == [3, 1]


def test_oracle_heads_and_tokens():
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(step.normed(x, np.array([1.0, 2.0]), 0.0), [[[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]]])
    y, size = step.rotated(x, [1], [np.pi / 2], True)
    assert np.allclose(y, [[[-4.0, 3.0]]]) and np.allclose(size, 7.0)
    c, s, _, h = step.quantise_tokens(np.array([[1.0, -0.5, 0.25, 0.0]], np.float16), 127)
    assert c.tolist() == [[127, -64, 32, 0]] and np.allclose(s, 1 / 127)          # 63.5: to the even one
    c, _, _, h = step.quantise_tokens(np.ones((1, 2), np.float16), 7, residual=np.array([[1.0, -3.0]], np.float16))
    assert h.tolist() == [[2.0, -2.0]] and c.tolist() == [[7, -7]]
    assert step.pack_int4(c).tolist() == [[0x97]]
    assert step.product(np.array([[1, 2]], np.int8), np.array([[3, 4]], np.int8), [0.5], [2.0]).tolist() == [[11.0]]
