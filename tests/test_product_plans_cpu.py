"""The plans of the dense product, as it describes them: the sizes that the GPU tests run reach every kernel, K split and
not, and incomplete tiles of each."""
import ctypes
import math
import random
import re

import pytest

import bit_unstructured_sparse_amd as bsp
from product_plans import COLUMNS, KERNELS, NEVER_SPLIT, ONE, SPLIT, STREAM


def plan(N, M, K, workspace):
    """(kernel, channels of a tile, tokens of a tile, splits)"""
    m = re.fullmatch(rf"dtype=int8 M={M} K={K} N={N} -> kernel=(.+) tile=(\d+)x(\d+) splits=(\d+)",
                     bsp.describe_gemm(M, K, N, workspace))
    return m[1], int(m[2]), int(m[3]), int(m[4])


def test_every_kernel_is_run_whole():
    seen = {}
    for N, M in ONE:
        for K in COLUMNS:
            kernel, channels, tokens, splits = plan(N, M, K, True)
            assert splits == 1 and plan(N, M, K, False) == (kernel, channels, tokens, 1)
            seen.setdefault(kernel, set()).add((M % channels > 0, N % tokens > 0, -(-M // 16) % (channels // 16) > 0))
    for N, M, K in STREAM:
        kernel, channels, tokens, splits = plan(N, M, K, True)
        assert splits == 1 and kernel.startswith("k_w8_stream")
        seen.setdefault(kernel, set()).add((M % 16 > 0, N % 16 > 0, False))
    assert sorted(seen) == sorted(KERNELS)
    for kernel, kinds in seen.items():
        assert any(k[0] for k in kinds) and any(k[1] for k in kinds), kernel
        # a tile with bands left over, where tiles have several
        assert any(k[2] for k in kinds) or kernel in KERNELS[:5] or kernel == "k_w8_ring<4, 1, 4, 3>", kernel


def test_every_kernel_is_run_split():
    seen = set()
    for N, M, K in SPLIT:
        kernel, channels, tokens, splits = plan(N, M, K, True)
        assert splits > 1 and M % channels and N % tokens and K % 64
        assert plan(N, M, K, False)[3] == 1
        seen.add(kernel)
    assert sorted(seen) == sorted(set(KERNELS) - set(NEVER_SPLIT))


def test_no_other_kernel_is_ever_chosen():
    rng = random.Random(5)
    log = lambda most: int(math.exp(rng.uniform(0, math.log(most))))
    for _ in range(20000):
        N, M, K = log(20000), log(200000), log(131071)
        for workspace in (False, True):
            kernel, _, _, splits = plan(N, M, K, workspace)
            assert kernel in KERNELS and (splits == 1 or (workspace and kernel not in NEVER_SPLIT))
            assert splits == 1 or bsp.gemm_workspace_bytes(M, K, N) > 0


def test_descriptions():
    L = bsp.load_library()
    buf = ctypes.create_string_buffer(256)
    assert L.gemm_w8a8_describe(64, 64, 4, 0, None, 256) == bsp.E_ARG and L.gemm_w8a8_describe(64, 64, 4, 0, buf, 0) == bsp.E_ARG
    for bad in ((-1, 64, 4), (64, -1, 4), (64, 64, -1)):
        assert L.gemm_w8a8_describe(*bad, 0, buf, 256) == bsp.E_ARG
    for bad in ((1 << 26, 64, 4), (64, 131072, 4), (64, 64, 1 << 31)):
        assert L.gemm_w8a8_describe(*bad, 0, buf, 256) == bsp.E_OVERFLOW
    for n in (1, 12, 60):      # cut off, and ended
        buf.raw = b"x" * 256
        assert L.gemm_w8a8_describe(4096, 4096, 8, 1, buf, n) == bsp.OK and len(buf.value) == n - 1 and buf.raw[n:n + 1] == b"x"
    assert bsp.describe_gemm(0, 64, 4) == "dtype=int8 M=0 K=64 N=4" and "kernel" not in bsp.describe_gemm(64, 64, 0)
    assert "kernel=k_w8_stream" in bsp.describe_gemm(64, 0, 4)
    # more tokens than a launch takes: its first run, not split
    assert "splits=1" in bsp.describe_gemm(1, 131071, 2 ** 31 - 1, workspace=True)
    with pytest.raises(bsp.BspError):
        bsp.describe_gemm(64, 131072, 4)
