"""Attention of drafted trees over the paged cache on the GPU, against the
oracle in 64 bits. The bound of each output follows from the arithmetic the
header states (tolerance(): nothing in it is fitted)."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import serving

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
KINDS = {"fp16": bsp.FP16, "int8": bsp.INT8, "int4": bsp.INT4}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def random_tree(rng, T):
    words = []
    for i in range(T):
        parent = int(rng.integers(-1, i)) if i else -1
        words.append((words[parent] if parent >= 0 else 0) | (1 << i))
    return np.array(words, np.uint64)


class Case:
    """B sequences with (T, len) each in a cache of shuffled pages; what no
    token uses holds NaN (fp16) or stale codes under NaN scale words."""

    def __init__(self, seed, lens, hq, hkv, D, kind, page, dev, tree=True, q_size=1.0, v_size=1.0, k_shift=0.5):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.hq, self.hkv, self.D, self.kind, self.page, self.dev = lens, hq, hkv, D, kind, page, dev
        B = len(lens)
        need = [-(-n // page) for _, n in lens]
        pages = sum(need) + 1
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((B, max(need + [1])), -7, np.int32)      # entries past a sequence are not read
        self.K, self.V, slots, at = [], [], [], 0
        for b, (T, n) in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            self.K.append((rng.normal(0, 1, (n, hkv, D)) + k_shift * rng.normal(0, 1, (1, hkv, D))).astype(np.float16))
            self.V.append((v_size * rng.normal(0, 1, (n, hkv, D))).astype(np.float16))
            j = np.arange(n)
            slots.append(self.table[b][j // page].astype(np.int64) * page + j % page if n else np.zeros(0, np.int64))
        c = bsp.new_kv_cache(KINDS[kind], pages, hkv, page, D, device=dev)
        if kind == "fp16":
            c.k.fill_(float("nan")), c.v.fill_(float("inf"))
        else:
            c.k.fill_(0xFF), c.v.fill_(0xC3)
            c.k_scale.fill_(serving.NAN_WORD), c.v_scale.fill_(0x7F807C00)      # NaN; infinite
        self.cache = c
        if at:
            bsp.kv_append(c, torch.from_numpy(np.concatenate(self.K)).to(dev),
                          torch.from_numpy(np.concatenate(self.V)).to(dev),
                          torch.from_numpy(np.concatenate(slots)).to(dev))
        self.slots = slots
        self.total = sum(T for T, _ in lens)
        self.Q = (q_size * rng.normal(0, 1, (self.total, hq, D))).astype(np.float16)
        self.masks = np.concatenate([random_tree(rng, T) for T, _ in lens] + [np.zeros(0, np.uint64)]) if tree else None
        self.scale = D ** -0.5

    def run(self, split=True, max_q=None, stream=None, Q=None, O=None, ws=None):
        d = self.dev
        mq = max([T for T, _ in self.lens] + [0]) if max_q is None else max_q
        table = torch.from_numpy(self.table).to(d)
        if split and ws is None:
            ws = bsp.new_attention_workspace(self.cache, len(self.lens), mq, self.hq, table.shape[1], device=d)
        self.ws = ws
        q_start = np.cumsum([0] + [T for T, _ in self.lens]).astype(np.int32)
        args = [torch.from_numpy(x).to(d) for x in (np.array([n for _, n in self.lens], np.int32), q_start)]
        mask = None if self.masks is None else torch.from_numpy(self.masks.view(np.int64)).to(d)
        Q = torch.from_numpy(self.Q).to(d) if Q is None else Q
        torch.cuda.synchronize()
        return bsp.attention_tree(Q, self.cache, table, *args, mq, tree_mask=mask, scale=self.scale, O=O,
                                  workspace=ws if split else None, stream=stream)

    def rows(self, name, b):
        """(values, reach) of sequence b's stored rows in 64 bits: reach bounds
        what the arithmetic on codes adds up in place of a value."""
        x = (self.K if name == "k" else self.V)[b]
        if self.kind == "fp16":
            return x.astype(np.float64), np.abs(x.astype(np.float64))
        s = self.slots[b]
        codes = getattr(self.cache, name).cpu().numpy()[s // self.page, :, s % self.page]
        words = getattr(self.cache, name + "_scale").cpu().numpy().view(np.uint32)[s // self.page, :, s % self.page]
        step, off = serving.unpack_word(words)
        v = serving.dequantise(codes, words, self.kind)
        return v, np.abs(v) + (step * serving.LEVELS[self.kind] + np.abs(off))[..., None]

    def expect(self):
        """(out, bound) [total][hq][D]."""
        G = self.hq // self.hkv
        out, tol = np.zeros(self.Q.shape), np.zeros(self.Q.shape)
        at = 0
        for b, (T, n) in enumerate(self.lens):
            if T == 0 or n == 0:
                at += T
                continue
            m = None if self.masks is None else self.masks[at:at + T]
            for name in ("k", "v"):
                setattr(self, name + "rows", self.rows(name, b))
            for h in range(self.hkv):
                q = self.Q[at:at + T, h * G:(h + 1) * G].astype(np.float64)
                (k, kr), (v, vr) = (tuple(y[:, h] for y in r) for r in (self.krows, self.vrows))
                o, _ = serving.attend(q, k, v, self.scale, m)
                _, spread = serving.attend(q, k, vr, self.scale, m)
                # a score: fp32 sums of D products of |q| and the reach of k
                dx = (self.D + 8) * 2.0 ** -24 * self.scale * np.abs(q).sum(-1).max() * kr.max()
                # weights: fp16 (2^-11) of a score off by dx, fp32 sums of n of them, small weights
                # cut off at 2^-30 of the scale, the result's own rounding
                bound = spread * (2.0 ** -11 + 2 * dx + (n + 64) * 2.0 ** -24) + np.abs(o) * 2.0 ** -11 + \
                    n * 2.0 ** -29 * vr.max() + 2.0 ** -24
                out[at:at + T, h * G:(h + 1) * G], tol[at:at + T, h * G:(h + 1) * G] = o, bound
            at += T
        return out, tol

    def check(self, O):
        torch.cuda.synchronize()
        got = O.cpu().numpy().astype(np.float64)
        want, tol = self.expect()
        assert np.isfinite(got).all()
        worst = np.abs(got - want) / tol
        assert worst.max(initial=0.0) <= 1.0, (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
        if self.ws is not None:
            assert not self.ws[:65536].any(), "an arrival counter was left behind"


LENS = [[(1, 1)], [(1, 16)], [(1, 17)], [(1, 500)], [(3, 3), (0, 40), (0, 0), (2, 65), (1, 129)],
        [(16, 16), (5, 300)], [(33, 100)], [(64, 64), (61, 333), (1, 31)], [(7, 1025), (1, 2100)]]


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "_".join(f"{t}x{n}" for t, n in v))
@pytest.mark.parametrize("split", [True, False])
def test_lengths(kind, lens, split, dev):
    c = Case(len(lens) + sum(n for _, n in lens), lens, 8, 2, 128, kind, 16, dev)
    c.check(c.run(split=split))


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("hq,hkv,D,page", [(1, 1, 64, 16), (5, 1, 64, 64), (3, 3, 128, 32), (16, 1, 128, 16),
                                           (20, 4, 128, 128), (17, 1, 256, 16), (8, 4, 256, 64), (40, 8, 64, 32)])
def test_heads_dims_pages(kind, hq, hkv, D, page, dev):
    c = Case(hq * 7 + D + page, [(6, 203), (1, 77), (13, 13)], hq, hkv, D, kind, page, dev)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("B,T,n", [(1, 1, 20000), (1, 12, 9001), (3, 2, 6007), (40, 1, 300)])
def test_long_and_many(kind, B, T, n, dev):
    c = Case(n, [(T, n - 97 * b) if n > 1000 else (T, n - 7 * b) for b in range(B)], 8, 2, 64, kind, 32, dev, tree=False)
    c.check(c.run())


def test_chain_without_a_mask_is_the_causal_mask(dev):
    c = Case(1, [(9, 50), (64, 64)], 4, 2, 64, "int8", 16, dev, tree=False)
    a = c.run()
    c.check(a)
    c.masks = np.concatenate([np.array([(2 << i) - 1 & (1 << 64) - 1 for i in range(T)], np.uint64) for T in (9, 64)])
    assert torch.equal(a, c.run())


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
def test_rows_that_see_nothing(kind, dev):
    c = Case(2, [(5, 5), (20, 23)], 4, 2, 64, kind, 16, dev)
    c.masks[[1, 4]] = 0            # no context and no drafted token: an empty row
    c.masks[6] = 0                 # the context alone
    O = c.run()
    c.check(O)
    assert not O[[1, 4]].any() and O[6].any()


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
def test_masked_rows_of_the_cache_have_no_effect(kind, dev):
    # a drafted token whose cache row is NaN or infinite: only the rows that see it may change
    c = Case(3, [(6, 40)], 4, 2, 128, kind, 16, dev)
    c.masks = np.array([0b1, 0b11, 0b101, 0b1001, 0b11011, 0b100001], np.uint64)
    base = c.run()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for j in (1, 3):
            t = torch.full((1, 2, 128), bad, dtype=torch.float16, device=dev)
            bsp.kv_append(c.cache, t, t, torch.from_numpy(c.slots[0][34 + j:35 + j]).to(dev))
        O = c.run()
        seen = [1, 3, 4]
        rest = [0, 2, 5]
        assert torch.equal(O[rest], base[rest])
        assert not torch.isfinite(O[seen]).any()


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("q_size,v_size", [(20.0, 1.0), (0.01, 1.0), (1.0, 4000.0), (4.0, 1e-3)])
def test_sharp_flat_large_small(kind, q_size, v_size, dev):
    c = Case(4, [(4, 700), (2, 33)], 8, 2, 128, kind, 16, dev, q_size=q_size, v_size=v_size)
    c.check(c.run())


@pytest.mark.parametrize("kind", ["fp16", "int8", "int4"])
def test_the_maximum_rises_along_the_sequence(kind, dev):
    # scores that grow towards the end, by far more than one rescaling step, and value
    # rows whose size grows with them and falls again
    c = Case(5, [(2, 900)], 4, 2, 64, kind, 16, dev)
    n = 900
    d = np.zeros((1, 1, 64), np.float16)
    d[..., 0] = 1
    c.K[0] = (c.K[0] * np.float16(0.2) + d * np.linspace(-30, 60, n)[:, None, None]).astype(np.float16)
    c.V[0] = (c.V[0] * np.where(np.arange(n) < 600, np.exp(np.arange(n) / 100.0), 0.01)[:, None, None]).astype(np.float16)
    c.Q[:] = np.abs(c.Q)
    bsp.kv_append(c.cache, *(torch.from_numpy(x[0]).to(dev) for x in (c.K, c.V)), torch.from_numpy(c.slots[0]).to(dev))
    c.check(c.run())


def test_strides_of_q_and_o(dev):
    c = Case(6, [(3, 50), (2, 20)], 4, 2, 64, "int8", 16, dev)
    want = c.run()
    for odd in (0, 3):
        wide = torch.full((5, 4 * 64 + 2 * 128 + odd), 7.0, dtype=torch.float16, device=dev)
        wide[:, odd:256 + odd] = torch.from_numpy(c.Q).to(dev).flatten(1)
        o = torch.full_like(wide, 5.0)
        c.run(Q=wide[:, odd:256 + odd].unflatten(1, (4, 64)), O=o[:, odd:256 + odd].unflatten(1, (4, 64)))
        torch.cuda.synchronize()
        assert torch.equal(o[:, odd:256 + odd].unflatten(1, (4, 64)), want)
        assert (o[:, 256 + odd:] == 5).all() and (o[:, :odd] == 5).all()


def test_workspace_reused_streams_and_repeats(dev):
    a = Case(7, [(1, 5000), (3, 2500)], 8, 2, 128, "int4", 16, dev)
    b = Case(8, [(20, 777)], 16, 2, 64, "fp16", 32, dev)
    oa, ob = a.run(), b.run()
    a.check(oa), b.check(ob)
    big = torch.zeros(max(a.ws.numel() if a.ws is not None else 0, b.ws.numel() if b.ws is not None else 0, 1 << 20),
                      dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for c, want in ((a, oa), (b, ob)):
            o = c.run(ws=big, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(o, want), "a repeat gave other bits"
    assert not big[:65536].any()


def test_graph_replays(dev):
    c = Case(9, [(2, 3000), (1, 100)], 8, 2, 128, "int8", 16, dev)
    want = c.run()
    table = torch.from_numpy(c.table).to(dev)
    kv, qs = torch.tensor([3000, 100], dtype=torch.int32, device=dev), torch.tensor([0, 2, 3], dtype=torch.int32, device=dev)
    mask, Q = torch.from_numpy(c.masks.view(np.int64)).to(dev), torch.from_numpy(c.Q).to(dev)
    ws, O = c.ws, torch.empty_like(want)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            bsp.attention_tree(Q, c.cache, table, kv, qs, 2, tree_mask=mask, scale=c.scale, O=O, workspace=ws)
    torch.cuda.synchronize()
    for _ in range(3):
        O.fill_(9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want)


def test_rows_past_max_q_and_unowned_rows_stay(dev):
    c = Case(10, [(5, 40), (2, 9)], 4, 2, 64, "int8", 16, dev, tree=False)
    O = torch.full((7, 4, 64), 3.0, dtype=torch.float16, device=dev)
    c.run(max_q=2, O=O)
    torch.cuda.synchronize()
    assert (O[2:5] == 3).all() and not (O[:2] == 3).all() and not (O[5:] == 3).all()


def test_offsets_past_32_bits(dev):
    # a cache of more than 4 GiB per tensor, the sequence's pages at its far end
    pages, hkv, page, D = 20500, 8, 64, 256
    c = bsp.KVCache(bsp.FP16, *(torch.zeros((pages, hkv, page, D), dtype=torch.float16, device=dev) for _ in "kv"))
    rng = np.random.default_rng(11)
    n = 100
    K, V = (rng.normal(0, 1, (n, hkv, D)).astype(np.float16) for _ in "kv")
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=dev)
    j = np.arange(n)
    slots = torch.from_numpy(np.array([pages - 1, pages - 3])[j // page] * page + j % page).to(dev)
    bsp.kv_append(c, torch.from_numpy(K).to(dev), torch.from_numpy(V).to(dev), slots)
    k, _ = bsp.kv_gather(c, slots)
    assert np.array_equal(k.cpu().numpy().view(np.uint16), K.view(np.uint16))
    Q = rng.normal(0, 1, (1, hkv, D)).astype(np.float16)
    O = bsp.attention_tree(torch.from_numpy(Q).to(dev), c, table, torch.tensor([n], dtype=torch.int32, device=dev),
                           torch.tensor([0, 1], dtype=torch.int32, device=dev), 1)
    torch.cuda.synchronize()
    for h in range(hkv):
        want, spread = serving.attend(Q[:, h:h + 1], K[:, h].astype(np.float64), V[:, h].astype(np.float64), D ** -0.5)
        assert (np.abs(O[:, h:h + 1].cpu().numpy() - want) <= 2.0 ** -10 * spread + 1e-4).all()


def test_python_refusals(dev):
    c = Case(12, [(2, 20)], 4, 2, 64, "int8", 16, dev)
    Q, cache = torch.from_numpy(c.Q).to(dev), c.cache
    table = torch.from_numpy(c.table).to(dev)
    one = torch.tensor([20], dtype=torch.int32, device=dev)
    qs = torch.tensor([0, 2], dtype=torch.int32, device=dev)
    ok = (Q, cache, table, one, qs, 2)
    assert bsp.attention_tree(*ok).shape == (2, 4, 64)

    def bad(exc, i, value, **kw):
        with pytest.raises(exc):
            bsp.attention_tree(*(value if i == j else a for j, a in enumerate(ok)), **kw)

    bad(TypeError, 0, Q.float())
    bad(TypeError, 0, Q.cpu())
    bad(ValueError, 0, Q[..., :32])
    bad(ValueError, 0, Q.transpose(0, 1))
    bad(bsp.BspError, 0, torch.cat([Q, Q[:, :1]], 1))          # 5 query heads over 2 kv heads
    bad(TypeError, 2, table.long())
    bad(ValueError, 2, table[0])
    bad(ValueError, 3, torch.zeros(2, dtype=torch.int32, device=dev))
    bad(ValueError, 4, one)
    bad(bsp.BspError, 5, 65)
    bad(TypeError, 9, None, tree_mask=torch.zeros(2, dtype=torch.int32, device=dev))
    bad(ValueError, 9, None, tree_mask=torch.zeros(3, dtype=torch.int64, device=dev))
    bad(ValueError, 9, None, O=torch.empty(3, 4, 64, dtype=torch.float16, device=dev))
    bad(bsp.BspError, 9, None, scale=float("nan"))
    bad(bsp.BspError, 9, None, workspace=torch.zeros(256, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        bsp.kv_append(cache, Q[:, :2], Q[:1, :2], torch.zeros(2, dtype=torch.int64, device=dev))
    with pytest.raises(TypeError):
        bsp.kv_append(cache, Q[:, :2], Q[:, :2], torch.zeros(2, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        bsp.KVCache(bsp.INT8, cache.k, cache.v, cache.k_scale[:1], cache.v_scale)
    with pytest.raises(ValueError):
        bsp.KVCache(bsp.FP16, cache.k.half(), cache.v.half(), cache.k_scale, None)
