"""Decode-step calls on a side stream while the current stream still has work:
the workspace and the outputs a call makes for itself are ordered with the
call, not with the current stream."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
import workloads

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _lora(dev, rng, M, K, N, R, kind):
    t = lambda x: torch.from_numpy(x).to(dev)
    ad = bsp.LoraAdapters(t((rng.normal(0, 1, (3, R, K)) / np.sqrt(K)).astype(np.float16)),
                          t((0.3 * rng.normal(0, 1, (3, M, R))).astype(np.float16)))
    index = t((np.arange(N) % 4 - 1).astype(np.int32))
    if kind == "f16":
        p = workloads.random_fp16_problem(M + N, M, K, N, 0.4)
        W, X = bsp.encode(p.W).to_device(dev), t(p.X)
        return lambda **kw: bsp.spmm_f16_lora(W, X, ad, index, **kw)
    p = workloads.random_int4_problem(M + N, M, K, N)
    W, X, X16 = bsp.encode(p.W).to_device(dev), t(bsp.pack_int4(p.X)), t(p.X.astype(np.float16))
    sw, sx = t(np.full(M, 1e-3, np.float32)), t(np.full(N, 0.5, np.float32))
    return lambda **kw: bsp.spmm_w4a4_dq_lora(W, X, X16, sw, sx, ad, index, **kw)


def _cache(dev, rng):
    cache = bsp.new_kv_cache(bsp.INT8, 40, 2, 16, 64, device=dev)
    rows = [torch.from_numpy(rng.normal(0, 1, (600, 2, 64)).astype(np.float16)).to(dev) for _ in "kv"]
    slots = torch.arange(600, device=dev)
    bsp.kv_append(cache, *rows, slots)
    return cache, slots


@pytest.mark.parametrize("call", ["f16_split", "f16", "w4a4_split", "w4a4", "gather", "attention"])
def test_side_stream_beside_a_busy_current_stream(call, dev):
    rng = np.random.default_rng(len(call))
    if call == "gather":
        cache, slots = _cache(dev, rng)
        fn = lambda **kw: torch.stack(bsp.kv_gather(cache, slots, **kw)) if not kw else bsp.kv_gather(cache, slots, **kw)
    elif call == "attention":
        cache, _ = _cache(dev, rng)
        i32 = dict(dtype=torch.int32, device=dev)
        Q = torch.from_numpy(rng.normal(0, 1, (3, 4, 64)).astype(np.float16)).to(dev)
        args = (Q, cache, torch.arange(40, **i32).view(1, 40), torch.tensor([600], **i32), torch.tensor([0, 3], **i32), 3)
        fn = lambda **kw: bsp.attention_tree(*args, **kw)
    else:
        kind, split = call.split("_")[0], call.endswith("split")
        M, K = (700, 11008) if kind == "f16" else (256, 16384)
        fn = _lora(dev, rng, M if split else 520, K if split else 1024, 8, 16, kind)
    want = fn()
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=dev, dtype=torch.float16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        for _ in range(8):
            busy = busy @ busy
        got = fn(stream=side)
        # blocks of the sizes a call asks for, on the current stream
        junk = [torch.full((n,), 7, dtype=torch.uint8, device=dev) for n in (65536, 1 << 18, 1 << 20, 1 << 21)]
        side.synchronize()
        torch.cuda.current_stream().wait_stream(side)
        got = torch.stack(got) if isinstance(got, tuple) else got
        assert torch.equal(got, want)
        del junk, got
    torch.cuda.synchronize()
