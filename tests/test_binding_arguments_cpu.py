"""What the native launch takes as an argument is what ctypes takes: a float or None for a number, None or bytes for a
factor and the like go to the Python function, which refuses them, and never reach an entry point as a zero. Without a
GPU, and in a process of its own: the native module has one set of functions to stand for."""
import subprocess
import sys

import pytest

import bit_unstructured_sparse_amd as bsp

SCRIPT = """
import ctypes, torch
import bit_unstructured_sparse_amd as bsp
from bit_unstructured_sparse_amd import _binding
L = bsp.load_library()
calls = []
def python(*args):
    calls.append(args)
    return "python"
_binding.bind(L._handle, {n: getattr(L, n) for n in bsp.EXPORTS}, (python,) * 5, torch)
names = ("kv_cache_append kv_cache_gather attention_tree_f16 kv_pages_step qk_norm_rope_f16 qk_norm_rope_append_f16 "
         "quantize_tokens_f16 dequantize_tokens_f16 gemm_w8a8_dq").split()
others = {ctypes.c_void_p: (2.0, "x", 1 << 64, 1j), ctypes.c_float: (None, b"x", "x", 1 << 64)}
tried = 0
for name in names:
    f = getattr(L, name)
    # zeros alone are refused, or launch nothing, before any HIP call
    fine = [0] * (len(f.argtypes) - 1)
    for i, t in enumerate(f.argtypes[:-1]):
        for bad in others.get(t, (2.0, 0.0, None, b"x", "x", 1 << 64)):
            args = fine[:i] + [bad] + fine[i + 1:]
            got = _binding.launch(f, 0, None, *args)
            assert got == "python" and calls.pop() == (f, 0, None, *args), (name, i, bad)
            tried += 1
print("tried", tried)
"""


def test_arguments_of_another_kind_go_to_python():
    pytest.importorskip("torch")
    pytest.importorskip("bit_unstructured_sparse_amd._binding")
    r = subprocess.run([sys.executable, "-c", SCRIPT], capture_output=True, text=True, timeout=300,
                       cwd=bsp.HERE.rsplit("/", 1)[0])
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout.split()[-1]) > 400
