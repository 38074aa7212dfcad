"""Heads and tokens at the sizes of prompts, where they are spread over wavefronts in other ways than in short calls: the
same bits as short calls, and the oracle's."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step
from test_gpu_heads import KINDS, _close, _fused
from test_gpu_tokens import _rows, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


# Heads of 128, 32768 of them and more: 8 rows a wavefront, of one kind where kinds fill them ((32, 32), and (31, 15) with
# the last wavefront of each kind filled in part), of several where they do not (5, 1). Heads of 64 and 256: 8 and 2 rows.
@pytest.mark.parametrize("D,n,hq,hkv", [(128, 700, 32, 32), (128, 701, 31, 15), (128, 3001, 28, 4), (128, 5500, 5, 1),
                                        (128, 33000, 1, 1), (64, 600, 32, 32), (64, 900, 23, 7), (64, 7000, 3, 1),
                                        (256, 300, 32, 16), (256, 1100, 9, 3), (256, 5000, 1, 1)])
@pytest.mark.parametrize("inter,part", [(False, 1), (True, 2)])
def test_heads(D, n, hq, hkv, inter, part, dev):
    rng = np.random.default_rng(D + n)
    rot = D // part
    wide, Q, K, V = _fused(rng, n, hq, hkv, D, 8, dev)
    positions = rng.integers(0, 1 << 20, n).astype(np.int32)
    pos = torch.from_numpy(positions).to(dev)
    w = [torch.from_numpy((1 + 0.3 * rng.normal(0, 1, D)).astype(np.float16)).to(dev) for _ in "qk"]
    freq = bsp.rope_frequencies(rot, device=dev)
    args = dict(q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=inter)
    q, k = bsp.qk_norm_rope(Q, K, pos, freq, **args)
    few = max(1, 30000 // (hq + 2 * hkv))
    for t in range(0, n, few):
        cut = slice(t, t + few)
        a, b = bsp.qk_norm_rope(Q[cut], K[cut], pos[cut], freq, **args)
        assert torch.equal(q[cut], a) and torch.equal(k[cut], b), t
    some = np.sort(rng.permutation(n)[:12])
    some[[0, -1]] = 0, n - 1
    for got, x, weight in ((q, Q, w[0]), (k, K, w[1])):
        _close(got[some], x[some].cpu().numpy(), weight.cpu().numpy(), 1e-5, positions[some], rot, inter)
    page, pages = 16, -(-n // 16) + 1
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[n // 3] = -1
    slots = torch.from_numpy(slots).to(dev)
    before = wide.clone()
    for kind in KINDS:
        one, two = (bsp.new_kv_cache(KINDS[kind], pages, hkv, page, D, device=dev) for _ in range(2))
        assert torch.equal(bsp.qk_norm_rope_append(Q, K, V, pos, freq, one, slots, **args), q)
        bsp.kv_append(two, k, V, slots)
        for name in ("k", "v", "k_scale", "v_scale"):
            a, b = getattr(one, name), getattr(two, name)
            assert (a is None and b is None) or torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (kind, name)
    assert torch.equal(wide, before)
    # in place: the results where the heads were, the rest as it was
    bsp.qk_norm_rope(Q, K, pos, freq, Qo=Q, Ko=K, **args)
    assert torch.equal(Q, q) and torch.equal(K, k)
    assert torch.equal(wide[:, (hq + hkv) * D:], before[:, (hq + hkv) * D:])


# 2048 tokens and more: two pieces a thread, a wavefront (up to 1024 channels) or four (up to 4096) a token
@pytest.mark.parametrize("dtype", [bsp.INT8, bsp.INT4])
@pytest.mark.parametrize("n", [2047, 2050])
@pytest.mark.parametrize("K", [513, 1000, 1024, 1025, 2048, 2049, 3001, 4096, 4097])
def test_tokens(dtype, n, K, dev):
    rng = np.random.default_rng(n + K)
    X = _rows(rng, n, K)
    weight = (1 + 0.2 * rng.normal(0, 1, K)).astype(np.float16)
    residual = rng.normal(0, 2, (n, K)).astype(np.float16)
    X[5, K - 1], X[1203, 0] = np.nan, np.inf
    x, w, r = (torch.from_numpy(a).to(dev) for a in (X, weight, residual))
    t = bsp.quantize_tokens(x, dtype, weight=w, eps=1e-5, residual=r, x16=True)
    finite = np.isfinite(X).all(1)
    rows = np.flatnonzero(finite)[::7]      # the oracle goes token by token
    pick = torch.from_numpy(rows).to(dev)
    check(bsp.Tokens(t.codes[pick], t.scale[pick], t.x16[pick], t.hidden[pick]), X[rows], dtype, weight, 1e-5, residual[rows], dev)
    assert torch.isnan(t.scale).cpu().numpy().tolist() == (~finite).tolist()
    for i in range(0, n, 500):
        s = bsp.quantize_tokens(x[i:i + 500], dtype, weight=w, eps=1e-5, residual=r[i:i + 500])
        assert torch.equal(t.codes[i:i + 500], s.codes)
        assert torch.equal(t.hidden[i:i + 500].view(torch.int16), s.hidden.view(torch.int16))
    back = bsp.dequantize_tokens(t.codes, t.scale, dtype, K)
    assert torch.equal(back[pick], bsp.dequantize_tokens(t.codes[pick], t.scale[pick], dtype, K))
    # the sum in place
    again = bsp.quantize_tokens(x, dtype, weight=w, eps=1e-5, residual=r, hidden=x)
    assert torch.equal(again.codes, t.codes) and torch.equal(x.view(torch.int16), t.hidden.view(torch.int16))
