"""Plain reference, in 64 bits and whole numbers, of the operators from a layer's
hidden states to the cache: the pages of a step, heads normed and rotated, tokens
quantised, the dense 8-bit product. Written from the definitions in
include/bitmap_spmm.h; shares no code with the library."""
import math
from fractions import Fraction

import numpy as np


class Pages:
    """Block tables and the list of free pages, one page at a time."""

    def __init__(self, table, lens, held, free, page_size):
        self.table = [list(r) for r in np.asarray(table).tolist()]
        self.lens, self.held = list(map(int, lens)), list(map(int, held))
        self.free = list(map(int, free))          # the pages of the list; the next to be taken last
        self.page = page_size

    def step(self, keep, new, rows, masks=None):
        """(slots, positions, sequences, q_start, kv_lens) of one step."""
        P, B = self.page, len(self.lens)
        width = len(self.table[0]) if B else 0
        first, keeps, wants = [0], [], []
        given = []
        for b in range(B):
            k = self.lens[b] if keep is None else min(max(int(keep[b]), 0), self.lens[b])
            m = max(int(new[b]), 0)
            keeps.append(k)
            first.append(first[b] + m)
            want = math.ceil(Fraction(k + m, P))
            if m and (first[-1] > rows or want > width):
                want = None                       # does not fit: waits
            wants.append(want)
            if want is not None and want < self.held[b]:
                given += self.table[b][want:self.held[b]]
        queue = list(given)
        stock = len(self.free) + len(given)
        asked = 0
        kv_lens = [0] * B
        slots, positions, sequences = [-1] * rows, [0] * rows, [-1] * rows
        for b in range(B):
            m = first[b + 1] - first[b]
            want = wants[b]
            if want is not None and want > self.held[b]:
                asked += want - self.held[b]
                if asked > stock:
                    want = None
                else:
                    for p in range(self.held[b], want):
                        self.table[b][p] = queue.pop(0) if queue else self.free.pop()
            self.lens[b] = keeps[b]
            if want is not None:
                self.held[b] = want
                self.lens[b] = kv_lens[b] = keeps[b] + m
            for i in range(m):
                r, t = first[b] + i, keeps[b] + i
                if r >= rows:
                    break
                sequences[r] = b
                positions[r] = t
                if masks is not None and m <= 64:
                    positions[r] = keeps[b] + sum(int(masks[r]) >> j & 1 for j in range(i))
                if want is not None:
                    slots[r] = self.table[b][t // P] * P + t % P
        self.free += queue[::-1]
        return slots, positions, sequences, [min(f, rows) for f in first], kv_lens


def normed(x, weight, eps):
    """Heads [..., D] in float64; weight None: as they are."""
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rotated(y, positions, angles, interleaved):
    """y [n][heads][D] rotated by positions[t] * angles[i] (radians, whole multiples of a turn taken out in exact
    arithmetic). Returns (result, size): size = |y1| + |y2| of the pair a channel belongs to."""
    y = np.array(y, np.float64)
    out, size = y.copy(), np.abs(y)
    half = len(angles)
    for t, p in enumerate(positions):
        for i, a in enumerate(angles):
            j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            turns = Fraction(int(p)) * Fraction(float(a) / (2.0 * math.pi))
            x = float(turns - math.floor(turns)) * 2.0 * math.pi
            c, s = math.cos(x), math.sin(x)
            out[t, :, j] = y[t, :, j] * c - y[t, :, k] * s
            out[t, :, k] = y[t, :, k] * c + y[t, :, j] * s
            size[t, :, j] = size[t, :, k] = np.abs(y[t, :, j]) + np.abs(y[t, :, k])
    return out, size


def quantise_tokens(X, levels, weight=None, eps=0.0, residual=None):
    """(codes int64 [n][K], scale float64 [n], y / sqrt(mean + eps) float64, hidden float16)."""
    h = np.asarray(X, np.float16)
    if residual is not None:
        with np.errstate(over="ignore", invalid="ignore"):
            h = (h.astype(np.float64) + np.asarray(residual, np.float16).astype(np.float64)).astype(np.float16)
    x = h.astype(np.float64)
    n, K = x.shape
    with np.errstate(invalid="ignore", over="ignore"):
        y = x if weight is None else x * np.asarray(weight, np.float16).astype(np.float64)
    codes, scale, x16 = np.zeros((n, K), np.int64), np.zeros(n), np.zeros((n, K))
    for t in range(n):
        with np.errstate(invalid="ignore", over="ignore"):
            d = 1.0 if weight is None else math.sqrt(np.dot(x[t], x[t]) / K + eps)
            x16[t] = y[t] / d if d != 0.0 else 0.0
        if not np.isfinite(y[t]).all():
            scale[t] = math.nan
            continue
        m = float(np.abs(y[t]).max())
        if m == 0.0:
            continue
        scale[t] = m / d / levels
        # 2 L |y| against odd multiples of m: both exact in 64 bits
        a = np.abs(y[t]) * (2 * levels)
        k = np.floor(a / (2 * m))
        border = (2 * k + 1) * m
        k = k + ((a > border) | ((a == border) & (k % 2 == 1)))
        codes[t] = (np.sign(y[t]) * k).astype(np.int64)
    return codes, scale, x16, h


def pack_int4(codes):
    """int [n][K] in [-8, 7] -> uint8 [n][ceil(K / 2)], low nibble first."""
    c = np.asarray(codes, np.int64) & 15
    if c.shape[1] % 2:
        c = np.concatenate((c, np.zeros((c.shape[0], 1), np.int64)), 1)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def product(W, X, scale_w, scale_x):
    """float16 [N][M]: exact sums, then fp32 factor by factor and one rounding to float16."""
    # float64 holds sums of fewer than 2^53 exactly
    s = X.astype(np.float64) @ W.astype(np.float64).T
    y = s.astype(np.float32) * np.asarray(scale_w, np.float32)[None, :] * np.asarray(scale_x, np.float32)[:, None]
    with np.errstate(over="ignore"):
        return y.astype(np.float16)
