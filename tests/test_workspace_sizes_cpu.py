"""Workspace sizes asked for before the nonzeros are known hold at every density."""
import random

import pytest

import bit_unstructured_sparse_amd as bsp

SHAPES = [(5792, 12183, 26), (5236, 10032, 24), (4096, 11008, 8), (2000, 16384, 32), (6000, 24576, 20)]


def _random_shapes(count):
    rng = random.Random(7)
    return [(int(2 ** rng.uniform(4, 15)), rng.randint(64, 30000), rng.randint(1, 32)) for _ in range(count)]


@pytest.mark.parametrize("dtype", [bsp.INT4, bsp.FP16])
def test_unknown_nonzeros(dtype):
    for M, K, N in SHAPES + _random_shapes(1500):
        most = bsp.workspace_bytes(dtype, M, K, N)
        lora = bsp.lora_workspace_bytes(dtype, M, K, N, 16)
        for i in range(0, 33, 2):
            nnz = M * K * i // 32
            assert bsp.workspace_bytes(dtype, M, K, N, nnz) <= most, (M, K, N, i)
            assert bsp.lora_workspace_bytes(dtype, M, K, N, 16, nnz) <= lora, (M, K, N, i)
