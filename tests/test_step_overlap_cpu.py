"""A step whose results would lie over what it reads is refused on the host, before any HIP call."""
import ctypes

import pytest

import bit_unstructured_sparse_amd as bsp

B, WIDTH, POOL, ROWS = 3, 4, 8, 10
# places 4 KiB apart: nothing overlaps
PLACES = ["block_table", "lens", "held", "free_pages", "keep", "new", "mask", "slots", "positions", "sequences", "q_start",
          "kv_lens"]
BYTES = dict(block_table=4 * B * WIDTH, lens=4 * B, held=4 * B, free_pages=4 * (2 + POOL), keep=4 * B, new=4 * B, mask=8 * ROWS,
             slots=8 * ROWS, positions=4 * ROWS, sequences=4 * ROWS, q_start=4 * (B + 1), kv_lens=4 * B)
OUTPUTS = ["slots", "positions", "sequences", "q_start", "kv_lens"]


def _call(**moved):
    at = dict({n: 0x100000 + 0x1000 * i for i, n in enumerate(PLACES)}, **moved)
    d = bsp._KVPagesDesc(B, WIDTH, 16, POOL, at["block_table"], at["lens"], at["held"], at["free_pages"])
    return bsp.load_library().kv_pages_step(ctypes.byref(d), at["keep"], at["new"], at["mask"], ROWS, at["slots"],
                                            at["positions"], at["sequences"], at["q_start"], at["kv_lens"], None)


@pytest.mark.parametrize("output", OUTPUTS)
def test_results_over_what_is_read_or_written(output):
    for other in PLACES:
        if other == output:
            continue
        here = 0x100000 + 0x1000 * PLACES.index(other)
        # the same place; its last 8 bytes; the result's last 8 bytes over its first
        for at in (here, here + (BYTES[other] - 8 & -8), here - (BYTES[output] - 8 & -8)):
            assert _call(**{output: at}) == bsp.E_ARG, (output, other, at - here)


def test_the_lengths_of_the_step_before():
    # out of the step before given again as out, its lengths as what is kept
    assert _call(keep=0x100000 + 0x1000 * PLACES.index("kv_lens")) == bsp.E_ARG
