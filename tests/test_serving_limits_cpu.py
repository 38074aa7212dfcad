"""Sizes at which the attention call's 32-bit indexes end: refused, or planned
without them, on the host. Nothing here reaches a GPU."""
import ctypes

import pytest

import bit_unstructured_sparse_amd as bsp

FAKE = 0x1000


def cache(page_size, head_dim=128, kv_heads=1):
    return bsp._KVCacheDesc(bsp.INT8, 8, kv_heads, page_size, head_dim, FAKE, FAKE, FAKE, FAKE)


def workspace(c, width, B, max_q, q_heads):
    n = ctypes.c_int64(-1)
    return bsp.load_library().attention_tree_workspace_bytes(ctypes.byref(c), width, B, max_q, q_heads, ctypes.byref(n)), n.value


def attend(c, width):
    """One sequence of one token, without a workspace; total_q 0 launches nothing."""
    return bsp.load_library().attention_tree_f16(FAKE, 128, ctypes.byref(c), FAKE, width, FAKE, FAKE, 1, 0, 1, 1, None,
                                                 0.1, FAKE, 128, None, 0, None)


@pytest.mark.parametrize("page", [16, 64, 4096])
def test_tokens_a_table_can_hold(page):
    # a lane looks 4 wavefronts x 31 tiles of 32 tokens, and its own tile, past the last
    most = (2 ** 31 - 1 - 4096) // page
    assert most * page + 4096 < 2 ** 31
    for width, status in ((most, bsp.OK), (most + 1, bsp.E_OVERFLOW), ((2 ** 31 - 1) // page, bsp.E_OVERFLOW)):
        assert attend(cache(page), width) == status
        assert workspace(cache(page), width, 1, 1, 1)[0] == status


def test_work_of_all_sequences_fits_32_bits():
    # 4 wavefronts side by side per tile of 32 tokens, and up to 512 chunks of
    # which the last is rounded up: past that a call is not split
    def work(width, B):
        return 4 * B * -(-width * 16 // 32)

    c = cache(16)
    for B in (9, 33, 512):
        most = (2 ** 31 - 1 - 512 * 16) // (4 * B) * 2
        for width, split in ((most, True), (most + 2, False)):
            assert (work(width, B) + 512 * 16 < 2 ** 31) == split
            rc, n = workspace(c, width, B, 64, 8)
            assert rc == bsp.OK and (n > 0) == split, (B, width, n)
    # sizes of calls are far from it
    assert workspace(c, 131072 // 16, 512, 64, 8)[1] > 0
