"""Calls through the native launch: numbers of another kind are refused as ctypes refuses them; several threads call on
the stream they share, and with a workspace of their own."""
import ctypes
import threading

import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    bsp._use_native()
    return torch.device("cuda:0")


@pytest.mark.parametrize("bad", [2.0, None, "2"])
def test_a_number_of_another_kind_is_refused(bad, dev):
    cache = bsp.new_kv_cache(bsp.FP16, 2, 1, 16, 64, device=dev)
    Q = torch.ones(2, 1, 64, dtype=torch.float16, device=dev)
    table, lens = (torch.zeros(1, n, dtype=torch.int32, device=dev) for n in (2, 1))
    start = torch.tensor([0, 2], dtype=torch.int32, device=dev)
    O = torch.full_like(Q, 5.0)
    with pytest.raises((ctypes.ArgumentError, TypeError)):
        bsp.attention_tree(Q, cache, table, lens.view(1), start, bad, O=O)
    pages = bsp.new_kv_pages(1, 2, 4, 16, device=dev)
    out = bsp.kv_step(pages, None, lens.view(1) + 2, 2)
    with pytest.raises((ctypes.ArgumentError, TypeError, ValueError)):
        bsp.kv_step(pages, None, lens.view(1), bad, out=out)
    torch.cuda.synchronize()
    assert (O == 5).all() and pages.lens.tolist() == [2]


def _threads(work, count=4):
    wrong = []

    def guarded(i):
        try:
            work(i)
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=guarded, args=(i,)) for i in range(count)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong


def test_several_threads_quantise_on_one_stream(dev):
    # outputs of one thread's calls are freed, and taken by another's, between the calls
    x = [torch.randn(100, 512, device=dev).half() for _ in range(4)]
    want = [bsp.quantize_tokens(a, bsp.INT8) for a in x]
    got = [None] * 4
    torch.cuda.synchronize()

    def work(i):
        for _ in range(50):
            got[i] = bsp.quantize_tokens(x[i], bsp.INT8)

    _threads(work)
    for a, b in zip(got, want):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)


def test_several_threads_multiply_on_one_stream(dev):
    # K split: parts and counters in a workspace of each thread's own
    rng = np.random.default_rng(4)
    enc = bsp.encode_int8(rng.integers(-128, 128, (512, 11008)).astype(np.int8), np.full(512, 1e-4, np.float32)).to_device(dev)
    X = torch.from_numpy(rng.integers(-128, 128, (400, 11008)).astype(np.int8)).to(dev)
    s = torch.full((400,), 0.01, device=dev)
    want = bsp.gemm_w8a8(enc, X, s)
    ws = [bsp.new_gemm_workspace(enc, 400, device=dev) for _ in range(4)]
    torch.cuda.synchronize()

    def work(i):
        for n in (400, 3, 65, 300, 33, 400):
            Y = bsp.gemm_w8a8(enc, X[:n], s[:n], workspace=ws[i])
            torch.cuda.current_stream().synchronize()
            assert torch.equal(Y, want[:n])

    _threads(work)
