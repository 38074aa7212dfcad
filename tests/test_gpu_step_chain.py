"""The operators from the hidden states to the cache together, as a served step uses them: pages of the step, tokens
normed and quantised, the fused projection, heads into the cache, attention over it, the output projection."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import serving, step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
HIDDEN, HQ, HKV, D, PAGE, B, ROWS, WIDTH = 256, 4, 2, 64, 16, 5, 24, 6


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


class Layer:
    """One attention layer over its own pages; sparse: the fused projection is the int4 sparse one."""

    def __init__(self, dev, sparse, kind, pool):
        rng = np.random.default_rng(11)
        M = (HQ + 2 * HKV) * D
        self.dev, self.sparse = dev, sparse
        self.sw = (0.02 * (0.5 + rng.random(M))).astype(np.float32)
        if sparse:
            self.W = (rng.integers(-8, 8, (M, HIDDEN)) * (rng.random((M, HIDDEN)) < 0.5)).astype(np.int8)
            self.proj = bsp.encode(self.W).to_device(dev)
        else:
            self.W = rng.integers(-127, 128, (M, HIDDEN)).astype(np.int8)
            self.sw = self.sw / 16
            self.proj = bsp.encode_int8(self.W, self.sw).to_device(dev)
        self.sw_dev = torch.from_numpy(self.sw).to(dev)
        self.out = bsp.encode_int8(rng.integers(-127, 128, (HIDDEN, HQ * D)).astype(np.int8),
                                   np.full(HIDDEN, 1e-4, np.float32)).to_device(dev)
        self.norm = torch.from_numpy((1 + 0.2 * rng.normal(0, 1, HIDDEN)).astype(np.float16)).to(dev)
        self.wq, self.wk = (torch.from_numpy((1 + 0.2 * rng.normal(0, 1, D)).astype(np.float16)).to(dev) for _ in "qk")
        self.freq = bsp.rope_frequencies(D, device=dev)
        self.cache = bsp.new_kv_cache(kind, 64, HKV, PAGE, D, device=dev)
        self.pages = bsp.new_kv_pages(B, WIDTH, pool, PAGE, device=dev)
        self.ws = bsp.new_attention_workspace(self.cache, B, 64, HQ, WIDTH, dev)

    def __call__(self, X, residual, keep, new, mask):
        s = bsp.kv_step(self.pages, keep, new, ROWS, tree_mask=mask)
        t = bsp.quantize_tokens(X, bsp.INT4 if self.sparse else bsp.INT8, weight=self.norm, eps=1e-5, residual=residual)
        if self.sparse:
            y = bsp.spmm_bitmap_w4a4_dq(self.proj, t.codes, ROWS, self.sw_dev, t.scale)
        else:
            y = bsp.gemm_w8a8(self.proj, t.codes, t.scale)
        y = y.view(ROWS, HQ + 2 * HKV, D)
        q = bsp.qk_norm_rope_append(y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:], s.positions, self.freq, self.cache,
                                    s.slots, q_weight=self.wq, k_weight=self.wk, eps=1e-5)
        O = torch.zeros_like(q)
        bsp.attention_tree(q, self.cache, self.pages.block_table, s.kv_lens, s.q_start, 64, tree_mask=mask, O=O,
                           workspace=self.ws)
        o = bsp.quantize_tokens(O.view(ROWS, HQ * D), bsp.INT8)
        return s, t, y, q, O, bsp.gemm_w8a8(self.out, o.codes, o.scale)


def _steps(rng):
    """(keep, new) of step after step: prompts, single tokens, drafts of which some are rejected, an end and a new prompt."""
    lens = np.zeros(B, int)
    for k in range(5):
        new = [[9, 1, 5, 0, 3], [1, 1, 1, 1, 1], [4, 4, 4, 4, 4], [2, 2, 2, 2, 2], [3, 3, 0, 3, 9]][k]
        keep = lens.copy()
        if k == 3:
            keep = np.maximum(keep - rng.integers(0, 4, B), 0)
        if k == 4:
            keep[2] = keep[4] = 0
        yield keep, np.array(new)
        lens = keep + new


@pytest.mark.parametrize("sparse,kind", [(False, bsp.FP16), (False, bsp.INT8), (True, bsp.INT4), (True, bsp.FP16)])
def test_steps_of_a_layer(sparse, kind, dev):
    rng = np.random.default_rng(5)
    layer = Layer(dev, sparse, kind, 64)
    name = {bsp.FP16: "fp16", bsp.INT8: "int8", bsp.INT4: "int4"}[kind]
    for keep, new in _steps(rng):
        X = rng.normal(0, 1, (ROWS, HIDDEN)).astype(np.float16)
        R = rng.normal(0, 2, (ROWS, HIDDEN)).astype(np.float16)
        used = int(new.sum())
        masks = np.zeros(ROWS, np.uint64)
        at = 0
        for m in new:
            for i in range(m):
                parent = int(rng.integers(-1, i)) if i else -1
                masks[at + i] = (int(masks[at + parent]) if parent >= 0 else 0) | (1 << i)
            at += m
        on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        s, t, y, q, O, out = layer(on(X), on(R), on(keep.astype(np.int32)), on(new.astype(np.int32)),
                                   on(masks.view(np.int64)))
        torch.cuda.synchronize()
        # each stage from what the one before it left
        codes, _, _, h = step.quantise_tokens(X, 7 if sparse else 127, layer.norm.cpu().numpy(), 1e-5, R)
        assert np.array_equal(t.hidden.cpu().numpy(), h)
        want = step.product(layer.W, codes, layer.sw, t.scale.cpu().numpy())
        assert np.array_equal(y.view(ROWS, -1).cpu().numpy(), want)
        positions = s.positions.cpu().numpy()
        depth = [bin(int(m) & ((1 << i) - 1)).count("1") for n in [0] for m, i in
                 zip(masks[:used], np.concatenate([np.arange(m) for m in new]))]
        assert positions[:used].tolist() == (np.repeat(keep, new) + depth).tolist()
        want, size = step.rotated(step.normed(y[:, :HQ].cpu().numpy(), layer.wq.cpu().numpy(), 1e-5), positions,
                                  10000.0 ** (-2.0 * np.arange(D // 2) / D), False)
        assert (np.abs(q.cpu().numpy() - want) <= np.abs(want) * 2.0 ** -11 + size * 2.0 ** -19 + 2.0 ** -25).all()
        # attention over the cache as it stands: the fp16 weights of the second product and the rounding of the result
        table = layer.pages.block_table.cpu().numpy()
        rows = lambda b, n, x: np.concatenate([x[table[b, p]] for p in range(max(1, -(-n // PAGE)))], 1)[:, :n]
        at = 0
        for b, m in enumerate(new):
            n = int(keep[b] + m)
            assert s.kv_lens[b] == n
            if n == 0:
                continue
            for h in range(HKV):
                kv = []
                for c, w in ((layer.cache.k, layer.cache.k_scale), (layer.cache.v, layer.cache.v_scale)):
                    a = rows(b, n, c.cpu().numpy())[h]
                    kv.append(a.astype(np.float64) if w is None else
                              serving.dequantise(a, rows(b, n, w.cpu().numpy().view(np.uint32)[..., None])[h][:, 0], name))
                G = HQ // HKV
                ref, spread = serving.attend(q[at:at + m, h * G:(h + 1) * G].cpu().numpy(), kv[0], kv[1], D ** -0.5,
                                             masks[at:at + m].tolist())
                got = O[at:at + m, h * G:(h + 1) * G].cpu().numpy().astype(np.float64)
                # weights rounded to 11 bits, a score's fp32 sum over 64 channels (under 2^-12 of a weight here)
                assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -10 + spread * 2.0 ** -9 + 2.0 ** -20).all()
            at += m
        assert not O[used:].any() and torch.isfinite(out).all()


def test_a_sequence_that_waits_gives_zeros_and_harms_nobody(dev):
    # one page for two sequences: the second waits, its rows give zeros, its slots are skipped
    layer = Layer(dev, False, bsp.FP16, 1)
    rng = np.random.default_rng(6)
    X = torch.from_numpy(rng.normal(0, 1, (ROWS, HIDDEN)).astype(np.float16)).to(dev)
    R = torch.zeros_like(X)
    new = torch.tensor([3, 2, 0, 0, 0], dtype=torch.int32, device=dev)
    s, _, _, _, O, _ = layer(X, R, None, new, None)
    assert s.kv_lens.tolist() == [3, 0, 0, 0, 0] and O[:3].any() and not O[3:].any()
    alone = layer.cache.k.clone()
    layer(X, R, new * 0, new, None)
    assert torch.equal(alone, layer.cache.k)


def test_captured_steps(dev):
    rng = np.random.default_rng(7)
    one, two = Layer(dev, True, bsp.INT8, 64), Layer(dev, True, bsp.INT8, 64)
    X, R = (torch.zeros(ROWS, HIDDEN, dtype=torch.float16, device=dev) for _ in "xr")
    keep, new = (torch.zeros(B, dtype=torch.int32, device=dev) for _ in "kn")
    one(X, R, keep, new, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one(X, R, keep, new, None)
    for k, n in _steps(rng):
        X.copy_(torch.from_numpy(rng.normal(0, 1, (ROWS, HIDDEN)).astype(np.float16)))
        R.copy_(torch.from_numpy(rng.normal(0, 2, (ROWS, HIDDEN)).astype(np.float16)))
        keep.copy_(torch.from_numpy(k.astype(np.int32))), new.copy_(torch.from_numpy(n.astype(np.int32)))
        graph.replay()
        want = two(X, R, keep, new, None)
        torch.cuda.synchronize()
        for a, b in zip(got[0] + got[1][:2] + got[2:], want[0] + want[1][:2] + want[2:]):
            assert torch.equal(a, b)
        assert torch.equal(one.cache.k, two.cache.k) and torch.equal(one.pages.free, two.pages.free)
