"""Plain numpy reference, in 64 bits, of the decode-step operators: the
quantised cache rows, attention of drafted trees over them, and adapters beside
a projection. Written from the definitions in include/bitmap_spmm.h; shares no
code with the library."""
import math

import numpy as np

LEVELS = {"int8": 255, "int4": 15}
NAN_WORD = 0x7FC07E00


def bfloat16_up(x: float) -> float:
    """The smallest bfloat16 (8 significant bits) at or above x >= 0."""
    if x == 0.0:
        return 0.0
    m, e = math.frexp(x)                      # x = m 2^e, 0.5 <= m < 1
    return math.ldexp(math.ceil(m * 256.0), e - 8)


def quantise_row(x, kind):
    """(codes, step, offset) of one row of float16 values."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros(x.size, np.int64), math.nan, math.nan
    L = LEVELS[kind]
    o = float(x.min())
    s = bfloat16_up(float(np.float32(x.max() - o) / np.float32(L)))
    if s == 0.0:
        return np.zeros(x.size, np.int64), 0.0, o
    u = np.minimum(np.rint((x - o) / s), L).astype(np.int64)
    return u, s, o


def word(step: float, offset: float) -> int:
    """The 32-bit scale word: bfloat16 step above float16 offset."""
    if math.isnan(step):
        return NAN_WORD
    hi = int(np.array(step, np.float32).view(np.uint32)) & 0xFFFF0000
    return hi | int(np.array(offset, np.float16).view(np.uint16))


def unpack_word(w):
    """(step, offset) as float64 arrays of uint32 words."""
    w = np.asarray(w).astype(np.uint32)
    step = (w & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
    off = (w & np.uint32(0xFFFF)).astype(np.uint16).view(np.float16).astype(np.float64)
    return step, off


def quantise(x, kind):
    """float16 rows [..., D] -> (code bytes as stored, words uint32)."""
    x = np.asarray(x, np.float16)
    flat = x.reshape(-1, x.shape[-1])
    codes = np.zeros(flat.shape, np.uint8)
    words = np.zeros(flat.shape[0], np.uint32)
    for i, row in enumerate(flat):
        u, s, o = quantise_row(row, kind)
        codes[i], words[i] = u, word(s, o)
    if kind == "int4":
        codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return codes.reshape(x.shape[:-1] + (-1,)), words.reshape(x.shape[:-1])


def dequantise(codes, words, kind):
    """What stored rows stand for, float64 [..., D]."""
    u = np.asarray(codes, np.uint8)
    if kind == "int4":
        u = np.stack((u & 15, u >> 4), -1).reshape(u.shape[:-1] + (-1,))
    s, o = unpack_word(words)
    return s[..., None] * u.astype(np.float64) + o[..., None]


def sees(i, j, past, T, mask):
    """Whether drafted token i sees token j (mask: its word, or None for a chain)."""
    d = j - past
    if d < 0:
        return True
    return d < T and (d <= i if mask is None else bool(int(mask) >> d & 1))


def attend(q, K, V, scale, masks=None):
    """Attention of one sequence and kv head in float64. q [T][G][D]; K, V
    [len][D]; masks: T words or None. Returns (out [T][G][D], spread [T][G][D]),
    spread = sum_j p_j |v_j|, zeros for rows that see nothing."""
    T, G, D = q.shape
    n = K.shape[0]
    out, spread = np.zeros((T, G, D)), np.zeros((T, G, D))
    for i in range(T):
        see = np.array([sees(i, j, n - T, T, None if masks is None else masks[i]) for j in range(n)], bool)
        if not see.any():
            continue
        k, v = K[see], V[see]
        x = (q[i].astype(np.float64) @ k.T) * scale
        e = np.exp(x - x.max(-1, keepdims=True))
        p = e / e.sum(-1, keepdims=True)
        out[i], spread[i] = p @ v, p @ np.abs(v)
    return out, spread


def lora(base, X, A, B, index, scale=None, rank=None):
    """base [N][M] + scale[a] B_a (A_a x_n) in float64."""
    Y = np.array(base, np.float64)
    R = A.shape[1]
    for n, a in enumerate(index):
        if a < 0 or a >= A.shape[0]:
            continue
        r = R if rank is None else int(min(max(rank[a], 0), R))
        t = A[a, :r].astype(np.float64) @ X[n].astype(np.float64)
        Y[n] += (1.0 if scale is None else float(scale[a])) * (B[a][:, :r].astype(np.float64) @ t)
    return Y
