"""Pins of the decode-step oracle (oracle/serving.py): hand-computed rows and
words, closed forms of attention, adapters against an explicit dense matrix."""
import numpy as np
import pytest

from oracle import serving


def test_bfloat16_up():
    assert serving.bfloat16_up(0.0) == 0.0
    assert serving.bfloat16_up(1.0) == 1.0
    assert serving.bfloat16_up(1.0 + 2.0 ** -20) == 1.0 + 2.0 ** -7      # 8 significant bits
    assert serving.bfloat16_up(255.5 * 2.0 ** -12) == 256.0 * 2.0 ** -12
    for x in np.random.default_rng(0).uniform(1e-6, 100.0, 200):
        y = serving.bfloat16_up(float(x))
        assert x <= y <= x * (1 + 2.0 ** -7)
        assert int(np.array(y, np.float32).view(np.uint32)) & 0xFFFF == 0


def test_rows_by_hand():
    # -1 .. 14 in steps of one: s = 1, o = -1, codes 0 .. 15
    u, s, o = serving.quantise_row(np.arange(-1, 15, dtype=np.float16), "int4")
    assert (s, o) == (1.0, -1.0) and u.tolist() == list(range(16))
    # half-way values go to the even code
    u, s, o = serving.quantise_row(np.array([0.0, 0.5, 1.5, 2.5, 15.0], np.float16), "int4")
    assert s == 1.0 and u.tolist() == [0, 0, 2, 2, 15]
    # a constant row: step zero, the offset is the value
    assert serving.quantise_row(np.full(4, -2.5, np.float16), "int8")[1:] == (0.0, -2.5)
    codes, words = serving.quantise(np.array([[0, 15, 1, 14]], np.float16), "int4")
    assert codes.tolist() == [[0xF0, 0xE1]] and words.tolist() == [0x3F800000]
    assert serving.quantise(np.array([[1.0, np.inf]], np.float16), "int8")[1].tolist() == [serving.NAN_WORD]


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_round_trip_within_half_a_step(kind):
    rng = np.random.default_rng(1)
    x = (rng.normal(0, 1, (50, 64)) * np.exp(rng.normal(0, 3, (50, 1)))).astype(np.float16)
    codes, words = serving.quantise(x, kind)
    s, o = serving.unpack_word(words)
    err = np.abs(serving.dequantise(codes, words, kind) - x.astype(np.float64))
    assert (err <= s[:, None] / 2 * (1 + 2.0 ** -20)).all()
    assert (o == x.min(-1)).all()


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    V = rng.normal(0, 1, (5, 4))
    q = np.zeros((2, 3, 4))
    out, _ = serving.attend(q, rng.normal(0, 1, (5, 4)), V, 0.5)
    assert np.allclose(out[0], V[:4].mean(0)) and np.allclose(out[1], V.mean(0))      # a chain: one token more
    out, spread = serving.attend(q, np.zeros((5, 4)), V, 1.0, masks=[0b01, 0b10])       # siblings
    assert np.allclose(out[1], V[[0, 1, 2, 4]].mean(0)) and np.allclose(spread[1], np.abs(V[[0, 1, 2, 4]]).mean(0))
    out, _ = serving.attend(q, np.full((2, 4), np.nan), np.full((2, 4), np.nan), 1.0, masks=[0, 0])
    assert (out == 0).all()                                                            # nothing seen
    # one token dominates
    K = np.zeros((5, 4))
    K[2, 0] = 1.0
    q[:, :, 0] = 100.0
    assert np.allclose(serving.attend(q, K, V, 1.0)[0], V[2])


def test_lora_is_a_dense_update():
    rng = np.random.default_rng(3)
    A, B, X = rng.normal(0, 1, (2, 8, 12)), rng.normal(0, 1, (2, 6, 8)), rng.normal(0, 1, (4, 12))
    W = rng.normal(0, 1, (6, 12))
    Y = serving.lora(X @ W.T, X, A, B, [1, -1, 0, 2], scale=[2.0, 0.5], rank=[3, 8])
    assert np.allclose(Y[0], (W + 0.5 * B[1] @ A[1]) @ X[0])
    assert np.allclose(Y[1], W @ X[1]) and np.allclose(Y[3], W @ X[3])
    assert np.allclose(Y[2], (W + 2.0 * B[0][:, :3] @ A[0][:3]) @ X[2])
