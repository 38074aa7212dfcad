"""Refusals of the decode-step entry points on the host: every call here fails
(or launches nothing) before any HIP call, the pointers are never dereferenced."""
import ctypes
import math

import pytest

import bit_unstructured_sparse_amd as bsp

FAKE = 0x1000


def cache(**kw):
    a = dict(dtype=bsp.INT8, num_pages=8, kv_heads=2, page_size=16, head_dim=64, k=FAKE, v=FAKE, k_scale=FAKE,
             v_scale=FAKE)
    a.update(kw)
    return bsp._KVCacheDesc(*(a[n] for n, _ in bsp._KVCacheDesc._fields_))


BAD_CACHES = [
    (dict(dtype=bsp.INT2), bsp.E_ARG), (dict(dtype=9), bsp.E_ARG), (dict(num_pages=-1), bsp.E_ARG),
    (dict(kv_heads=-1), bsp.E_ARG), (dict(page_size=8), bsp.E_ARG), (dict(page_size=48), bsp.E_ARG),
    (dict(page_size=8192), bsp.E_ARG), (dict(head_dim=96), bsp.E_UNSUPPORTED), (dict(head_dim=0), bsp.E_UNSUPPORTED),
    (dict(num_pages=1 << 28), bsp.E_OVERFLOW), (dict(kv_heads=1 << 16), bsp.E_OVERFLOW), (dict(k=None), bsp.E_ARG),
    (dict(v=None), bsp.E_ARG), (dict(k=FAKE + 8), bsp.E_ARG), (dict(k_scale=None), bsp.E_ARG),
    (dict(v_scale=FAKE + 4), bsp.E_ARG),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_cache_descriptors(bad, status):
    L, c = bsp.load_library(), cache(**bad)
    assert L.kv_cache_append(ctypes.byref(c), FAKE, 128, FAKE, 128, FAKE, 4, None) == status
    assert L.kv_cache_gather(ctypes.byref(c), FAKE, 4, FAKE, 128, FAKE, 128, None) == status
    n = ctypes.c_int64(-1)
    assert L.attention_tree_workspace_bytes(ctypes.byref(c), 4, 1, 1, 2, ctypes.byref(n)) in (status, bsp.E_ARG)


@pytest.mark.parametrize("fn", ["kv_cache_append", "kv_cache_gather"])
def test_cache_calls(fn):
    L, c = bsp.load_library(), cache()

    def call(c=c, K=FAKE, ks=128, V=FAKE, vs=128, slots=FAKE, n=4):
        r = None if c is None else ctypes.byref(c)
        if fn == "kv_cache_append":
            return L.kv_cache_append(r, K, ks, V, vs, slots, n, None)
        return L.kv_cache_gather(r, slots, n, K, ks, V, vs, None)

    assert call(c=None) == bsp.E_ARG
    for bad in (dict(n=-1), dict(K=None), dict(V=None), dict(slots=None), dict(ks=127), dict(vs=0), dict(K=FAKE + 1),
                dict(slots=FAKE + 4)):
        assert call(**bad) == bsp.E_ARG, bad
    assert call(n=1 << 40) == bsp.E_OVERFLOW and call(n=1 << 27) == bsp.E_OVERFLOW
    assert call(n=0, K=None) == bsp.OK and call(c=cache(kv_heads=0, k=None, v=None)) == bsp.OK
    if fn == "kv_cache_append":
        assert call(c=cache(num_pages=0, k=None, v=None, k_scale=None, v_scale=None)) == bsp.OK   # every slot is outside


def test_attention_calls():
    L = bsp.load_library()
    base = dict(Q=FAKE, qs=8 * 64, c=cache(), table=FAKE, width=4, lens=FAKE, start=FAKE, B=3, total=9, max_q=4, hq=8,
                mask=None, scale=0.1, O=FAKE, os=8 * 64, ws=None, wb=0)

    def call(**kw):
        a = dict(base, **kw)
        c = None if a["c"] is None else ctypes.byref(a["c"])
        return L.attention_tree_f16(a["Q"], a["qs"], c, a["table"], a["width"], a["lens"], a["start"], a["B"],
                                    a["total"], a["max_q"], a["hq"], a["mask"], a["scale"], a["O"], a["os"], a["ws"],
                                    a["wb"], None)

    for bad in (dict(c=None), dict(Q=None), dict(O=None), dict(lens=None), dict(start=None), dict(table=None),
                dict(width=-1), dict(B=-1), dict(total=-1), dict(max_q=-1), dict(max_q=65), dict(hq=7), dict(hq=-2),
                dict(qs=8 * 64 - 1), dict(os=0), dict(Q=FAKE + 1), dict(mask=FAKE + 4), dict(scale=math.inf),
                dict(scale=math.nan), dict(scale=1e39), dict(wb=256), dict(ws=FAKE + 16, wb=1 << 30), dict(wb=-1),
                dict(c=cache(kv_heads=0)), dict(c=cache(num_pages=0))):
        assert call(**bad) == bsp.E_ARG, bad
    assert call(c=cache(head_dim=80)) == bsp.E_UNSUPPORTED
    assert call(hq=2 * 16400, qs=1 << 24, os=1 << 24) == bsp.E_UNSUPPORTED
    for bad in (dict(B=1 << 17), dict(hq=1 << 17), dict(total=1 << 33), dict(width=1 << 30)):
        assert call(**bad) == bsp.E_OVERFLOW, bad
    assert call(ws=FAKE, wb=256) == bsp.E_CAPACITY
    for none in (dict(B=0), dict(max_q=0), dict(total=0), dict(hq=0)):
        assert call(**none, Q=None, O=None) == bsp.OK, none


def test_attention_workspace():
    L, n = bsp.load_library(), ctypes.c_int64(-1)
    size = lambda c, *a: (L.attention_tree_workspace_bytes(ctypes.byref(c), *a, ctypes.byref(n)), n.value)
    assert L.attention_tree_workspace_bytes(ctypes.byref(cache()), 4, 1, 1, 2, None) == bsp.E_ARG
    assert size(cache(), 4, 0, 1, 2) == (bsp.OK, 0) and size(cache(), 4, 1, 0, 2) == (bsp.OK, 0)
    rc, short = size(cache(), 4, 1, 1, 2)
    rc2, long = size(cache(), 4096, 1, 1, 2)
    assert rc == rc2 == bsp.OK and 65536 < short < long
    # the parts of one round of workgroups, whatever the lengths are
    assert size(cache(), 1 << 20, 64, 64, 64)[1] < 1 << 27
    assert size(cache(), 4, 1, 1, 3)[0] == bsp.E_ARG


def test_lora_calls():
    L = bsp.load_library()
    ok = dict(adapters=2, rank=16, A=FAKE, B=FAKE, scale=None, ranks=None, index=FAKE)

    def f16(ws=None, wb=0, M=64, K=64, X=FAKE, N=2, Y=FAKE, **kw):
        d = bsp._LoraDesc(*(dict(ok, **kw)[n] for n, _ in bsp._LoraDesc._fields_))
        return L.spmm_bitmap_f16_lora(FAKE, FAKE, FAKE, 64, M, K, X, N, ctypes.byref(d), Y, ws, wb, None)

    def dq(ws=None, wb=0, sw=FAKE, sx=FAKE, X16=FAKE, **kw):
        d = bsp._LoraDesc(*(dict(ok, **kw)[n] for n, _ in bsp._LoraDesc._fields_))
        return L.spmm_bitmap_w4a4_dq_lora(FAKE, FAKE, FAKE, 64, 64, 64, FAKE, X16, 2, sw, sx, ctypes.byref(d), FAKE, ws,
                                          wb, None)

    for bad in (dict(adapters=-1), dict(rank=0), dict(rank=12), dict(rank=264), dict(A=None), dict(B=None),
                dict(A=FAKE + 8), dict(B=FAKE + 2), dict(index=None), dict(wb=-1), dict(wb=64),
                dict(ws=FAKE + 16, wb=1 << 20)):
        assert f16(**bad) == bsp.E_ARG, bad
        assert dq(**bad) == bsp.E_ARG, bad
    assert f16(adapters=1 << 33) == bsp.E_OVERFLOW
    assert f16() == bsp.E_CAPACITY and f16(ws=FAKE, wb=256) == bsp.E_CAPACITY and dq() == bsp.E_CAPACITY
    assert f16(X=None) == bsp.E_ARG and f16(Y=None) == bsp.E_ARG and f16(N=33) == bsp.E_ARG
    assert dq(sw=None) == bsp.E_ARG and dq(sx=None) == bsp.E_ARG and dq(X16=None) == bsp.E_ARG
    assert f16(N=0) == bsp.OK and f16(M=0) == bsp.OK
    assert L.spmm_bitmap_f16_lora(FAKE, FAKE, FAKE, 64, 64, 64, FAKE, 2, None, FAKE, None, 0, None) == bsp.E_ARG


def test_lora_workspace():
    # the counters, t, and (int4) the int32 sums; more where the projection splits K
    assert bsp.lora_workspace_bytes(bsp.FP16, 512, 64, 3, 16) >= 65536 + 3 * 16 * 4
    assert bsp.lora_workspace_bytes(bsp.INT4, 512, 64, 3, 16) >= 65536 + 3 * 16 * 4 + 512 * 3 * 4
    assert bsp.lora_workspace_bytes(bsp.FP16, 4096, 11008, 8, 16) > bsp.workspace_bytes(bsp.FP16, 4096, 11008, 8)
    assert bsp.lora_workspace_bytes(bsp.FP16, 0, 64, 3, 16) == 0
    for bad in ((bsp.FP16, 64, 64, 33, 16), (bsp.FP16, 64, 64, 1, 4), (bsp.INT2, 64, 64, 1, 8), (bsp.FP16, -1, 64, 1, 8)):
        with pytest.raises(bsp.BspError):
            bsp.lora_workspace_bytes(*bad)


def test_python_refuses_what_is_not_on_the_device():
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        bsp.KVCache(bsp.INT8, t, t, t, t)
    with pytest.raises(ValueError):
        bsp.KVCache(bsp.INT2, t, t, t, t)
    with pytest.raises(ValueError):
        bsp.new_kv_cache(7, 1, 1, 16, 64)
    a = torch.zeros(1, 8, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        bsp.LoraAdapters(a, torch.zeros(1, 32, 16, dtype=torch.float16))
    with pytest.raises(TypeError):
        bsp.LoraAdapters(a, torch.zeros(1, 32, 8, dtype=torch.float16))
