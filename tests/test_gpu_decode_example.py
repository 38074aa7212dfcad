"""The decode-step example: projection with adapters, cache, tree attention and
output projection together, eager and replayed, against its 64-bit reference."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")


@pytest.mark.parametrize("cache", ["fp16", "int8", "int4"])
@pytest.mark.parametrize("size", [dict(hidden=512, heads=8, kv_heads=2, head_dim=64, batch=3, tree=5, context=77),
                                  dict(hidden=640, heads=4, kv_heads=4, head_dim=128, batch=1, tree=1, context=300),
                                  dict(hidden=256, heads=6, kv_heads=1, head_dim=256, batch=2, tree=16, context=33)])
def test_example(cache, size):
    spec = importlib.util.spec_from_file_location("decode_step", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    argv = [f"--{k.replace('_', '-')}={v}" for k, v in size.items()]
    error, moved = ex.main(argv + ["--cache", cache, "--steps", "3", "--page", "16"])
    # The query, the attention and the result are each rounded to fp16 on both
    # sides and may fall on neighbouring values, the softmax weights once more:
    # four half-ulps, times the spread of a sum over the projection (under 8).
    assert error < 4 * 2.0 ** -11 * 8
    # Rows within +-8 (normal draws of unit size, projections of them) quantised
    # anew: at most one step of 16 / L, and its bfloat16 rounding.
    assert moved <= {"fp16": 0.0, "int8": 16 / 255, "int4": 16 / 15}[cache] * (1 + 2.0 ** -7)
