"""Value rows of very different steps in a quantised cache: a row counts in the
arithmetic with its weight, so that a large one a query row does not see, or
sees with no weight to speak of, costs the others nothing."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import serving
from test_gpu_attention_tree import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def put(c, b, tokens):
    """Write sequence b's K and V rows of these tokens into the cache again."""
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x[b][tokens])).to(c.dev)
    bsp.kv_append(c.cache, t(c.K), t(c.V), torch.from_numpy(c.slots[b][tokens]).to(c.dev))


def check(c, O):
    """Every output within what the arithmetic on the tokens its row sees allows:
    fp16 weights (2^-11 each) of scores off by dx (a token's own), fp32 sums, the result's own
    rounding, and weight times step cut off at half of the least fp16 number,
    2^-31 of the largest the row has, times the largest code."""
    torch.cuda.synchronize()
    got = O.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    G, at, worst = c.hq // c.hkv, 0, 0.0
    L = serving.LEVELS[c.kind]
    for b, (T, n) in enumerate(c.lens):
        k, kr = c.rows("k", b)
        v, vr = c.rows("v", b)
        words = c.cache.v_scale.cpu().numpy().view(np.uint32)[c.slots[b] // c.page, :, c.slots[b] % c.page]
        step = serving.unpack_word(words)[0]
        for i in range(T):
            see = np.array([serving.sees(i, j, n - T, T, c.masks[at + i]) for j in range(n)])
            for h in range(c.hq):
                g = h // G
                q = c.Q[at + i, h].astype(np.float64)
                x = k[see, g] @ q * c.scale
                p = np.exp(x - x.max())
                p /= p.sum()
                want, spread = p @ v[see, g], p @ vr[see, g]
                dx = (c.D + 8) * 2.0 ** -24 * c.scale * np.abs(q).sum() * kr[see, g].max(-1)
                tol = spread * (2.0 ** -11 + 2 * (p @ dx) + (n + 64) * 2.0 ** -24) + 2 * (p * dx) @ vr[see, g] + \
                    np.abs(want) * 2.0 ** -11 + n * 2.0 ** -31 * L * (p * step[see, g]).max() + 2.0 ** -24
                worst = max(worst, (np.abs(got[at + i, h] - want) / tol).max())
        at += T
    assert worst <= 1.0, worst


SIZES = [(1e-1, 500), (1e-2, 500), (2e-3, 500), (1e-2, 3000)]


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("size,n", SIZES)
@pytest.mark.parametrize("hq", [2, 24])
def test_a_large_row_that_is_not_seen(kind, size, n, hq, dev):
    c = Case(n + hq, [(4, n)], hq, 2, 128, kind, 16, dev, v_size=size)
    c.masks = np.array([0b1, 0b11, 0b101, 0b1101], np.uint64)        # token 1 is seen by itself alone
    base = c.run()
    check(c, base)
    c.V[0][n - 3] = np.where(np.arange(128) % 2, 6e4, -6e4)
    put(c, 0, [n - 3])
    O = c.run()
    check(c, O)
    assert torch.equal(O[[0, 2, 3]], base[[0, 2, 3]]), "a row that is not seen has an effect"


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("size,n,at", [(size, n, at) for size, n in SIZES for at in (0, 200, 499)] +
                         [(size, n, at) for size, n in ((1e-3, 20), (3e-4, 20), (3e-4, 2)) for at in (0, 1)])
def test_a_large_row_of_no_weight(kind, size, n, at, dev):
    # the key of token `at` points away from every query: scores of -100 and less
    c = Case(n + at, [(1, n)], 8, 2, 128, kind, 16, dev, v_size=size)
    c.Q[..., 0] = 8.0
    c.K[0][..., 0] = 0.0
    c.K[0][at, :, 0] = -400.0
    c.V[0][at] = np.where(np.arange(128) % 2, 3e4, -3e4)
    put(c, 0, np.arange(n))
    check(c, c.run())
    check(c, c.run(split=False))


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("split", [True, False])
def test_steps_that_grow_fall_and_are_zero(kind, split, dev):
    # sizes over 2^24, rows of one value (step 0) and of zeros, first and last
    n = 1200
    c = Case(77, [(3, n), (1, 40), (2, 2)], 8, 2, 64, kind, 32, dev)
    for b, (_, m) in enumerate(c.lens):
        j = np.arange(m)
        size = 2.0 ** (12 * np.sin(j / 37.0))
        c.V[b] = (np.clip(c.V[b] * size[:, None, None], -6e4, 6e4)).astype(np.float16)
        c.V[b][j % 5 == 0] = 0.0
        c.V[b][j % 7 == 0] = np.float16(-3.5)
        put(c, b, j)
    check(c, c.run(split=split))
    for b, (_, m) in enumerate(c.lens):
        c.V[b][:] = np.float16(0.75)          # every step is zero
        put(c, b, np.arange(m))
    O = c.run(split=split)
    check(c, O)
    assert (O == 0.75).all()
