"""Infinities and NaN in single channels of an fp16 cache's value rows: by the
definition they reach that channel of the rows that see the token, wherever it
lies in the sequence, and nothing else."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import serving
from test_gpu_attention_tree import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def check(c, bad, **run):
    """bad: (sequence, token, kv head, channel, value) put into V. The finite
    channels are those of zeros in their place, the others sums of what is seen."""
    clean = [x.copy() for x in c.V]
    for b, j, g, d, value in bad:
        c.V[b][j, g, d] = value
        clean[b][j, g, d] = 0.0
    for b in range(len(c.lens)):
        t = lambda x: torch.from_numpy(x[b]).to(c.dev)
        bsp.kv_append(c.cache, t(c.K), t(c.V), torch.from_numpy(c.slots[b]).to(c.dev))
    O = c.run(**run)
    torch.cuda.synchronize()
    got = O.cpu().numpy().astype(np.float64)
    c.V = clean
    want, tol = c.expect()
    G, at, odd = c.hq // c.hkv, 0, np.zeros(want.shape)
    for b, (T, n) in enumerate(c.lens):
        for bb, j, g, d, value in bad:
            for i in range(T):
                if bb == b and serving.sees(i, j, n - T, T, None if c.masks is None else c.masks[at + i]):
                    with np.errstate(invalid="ignore"):          # inf - inf
                        odd[at + i, g * G:(g + 1) * G, d] += value
        at += T
    finite = np.isfinite(odd)
    assert np.array_equal(got[~finite], odd[~finite], equal_nan=True)
    assert np.isfinite(got[finite]).all(), "a channel without an infinity is not finite"
    assert (np.abs(got - want)[finite] <= tol[finite]).all()


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("at", [0, 31, 32, 63, 64, 90, 96])
@pytest.mark.parametrize("hq,D", [(2, 64), (2, 128), (16, 128), (6, 256)])
def test_one_channel_of_a_context_row(value, at, hq, D, dev):
    c = Case(at + D + hq, [(3, 100), (1, 40)], hq, 2, D, "fp16", 16, dev)
    check(c, [(0, at, 1, 5, value)])


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("hq,D", [(2, 64), (16, 128), (6, 256)])
def test_one_channel_of_a_drafted_row(value, hq, D, dev):
    c = Case(D + hq, [(4, 70), (2, 2)], hq, 2, D, "fp16", 16, dev)
    c.masks = np.array([0b1, 0b11, 0b101, 0b1101, 0b1, 0b10], np.uint64)
    check(c, [(0, 67, 0, D - 1, value), (0, 68, 1, 0, value), (1, 0, 1, 17, value)])


@pytest.mark.parametrize("split", [True, False])
def test_both_signs_and_several_rows(split, dev):
    # one sign in one channel, both in another, in one tile and over several
    c = Case(3, [(9, 2000), (2, 50), (1, 33)], 16, 2, 128, "fp16", 32, dev)
    check(c, [(0, 1990, 0, 3, INF), (0, 1980, 0, 3, INF), (0, 1981, 0, 4, INF), (0, 1982, 0, 4, -INF), (0, 7, 1, 9, INF),
              (0, 1991, 1, 9, -INF), (1, 48, 1, 127, -INF), (1, 49, 1, 127, NAN), (2, 31, 0, 64, INF), (2, 32, 0, 65, -INF)],
          split=split)
