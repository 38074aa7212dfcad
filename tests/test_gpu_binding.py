"""The binding's native steps: what they accept and give is what the Python functions they stand for accept and
give, and every other case goes to those."""
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


@pytest.fixture(scope="module")
def native():
    from bit_unstructured_sparse_amd import _binding
    return _binding


def _python(name):
    """The function as written in Python."""
    import importlib.util
    spec = importlib.util.spec_from_file_location("bsp_plain", bsp.__file__)
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["bsp_plain"] = m
    spec.loader.exec_module(m)
    return getattr(m, name)


def _outcome(f, *args):
    try:
        return f(*args)
    except Exception as e:
        return type(e).__name__, str(e)


def test_native_steps_are_in_use(dev, native):
    assert bsp._flat is native.flat and bsp._launch is native.launch and bsp._new_output is native.new_output


def test_checks_agree(dev, native):
    h = torch.zeros(6, 4, 64, dtype=torch.float16, device=dev)
    wide = torch.zeros(6, 10, 64, dtype=torch.float16, device=dev)
    tensors = [h, wide[:, :4], wide[:, 1:5], wide[:1, :4], wide[::2, :4], h.transpose(0, 1), h.transpose(1, 2), h[:, :, ::2],
               h.float(), h.cpu(), h[:0], h.flatten(), wide[:, :1], wide.expand(6, 10, 64), h[:1].expand(6, 4, 64),
               h.view(6, 256), wide.view(6, 640)[:, :256], h.view(6, 256).t(), torch.zeros(6, 0, device=dev).half(), None, 3, "x",
               torch.nn.Parameter(h, requires_grad=False), torch.zeros(24, 64, dtype=torch.float16, device=dev)]
    flat, rows, matrix = _python("_flat"), _python("_rows"), _python("_matrix_rows")
    f16 = torch.float16
    for t in tensors:
        for numel in (1536, 384, 0, 64):
            for index in (0, 1):
                a = (t, "t", f16, numel, index)
                assert _outcome(native.flat, *a) == _outcome(flat, *a), a
        for n in (None, 6, 1, 0, 3):
            for heads, dim in ((4, 64), (1, 64), (4, 32), (10, 64)):
                a = (t, "t", n, heads, dim, 0)
                assert _outcome(native.rows, *a) == _outcome(rows, *a), a
        for n in (6, 0, 24):
            for width in (256, 64, 0, 6):
                a = (t, "t", f16, n, width, 0)
                assert _outcome(native.matrix_rows, *a) == _outcome(matrix, *a), a
    assert _outcome(native.flat, h, "t", torch.float32, 1536, 0) == _outcome(flat, h, "t", torch.float32, 1536, 0)


def test_outputs(dev, native):
    for shape, dtype in (((3, 4), torch.float16), ((0,), torch.int32), ((2, 3, 4), torch.int64), ((5, 0), torch.uint8)):
        t = native.new_output(shape, dtype, dev, None)
        assert t.shape == shape and t.dtype == dtype and t.device == dev and t.is_contiguous()
    side = torch.cuda.Stream()
    t = native.new_output((8,), torch.int32, dev, side)
    assert t.shape == (8,) and t.device == dev
    with pytest.raises((RuntimeError, TypeError)):
        native.new_output((-1,), torch.int32, dev, None)


def test_a_call_on_the_current_stream_or_another(dev):
    x = torch.randn(64, 256, device=dev).half()
    want = bsp.quantize_tokens(x, bsp.INT8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = bsp.quantize_tokens(x, bsp.INT8)
    b = bsp.quantize_tokens(x, bsp.INT8, stream=side)
    torch.cuda.synchronize()
    for t in (a, b):
        assert torch.equal(t.codes, want.codes) and torch.equal(t.scale, want.scale)
    # captured: the native launch goes to the capturing stream
    codes, scale = torch.zeros_like(want.codes), torch.zeros_like(want.scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsp.quantize_tokens(x, bsp.INT8, codes=codes, scale=scale)
    assert not codes.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(codes, want.codes)


def test_refusals_reach_the_caller(dev):
    x = torch.zeros(2, 64, dtype=torch.float16, device=dev)
    with pytest.raises(bsp.BspError) as e:
        bsp.quantize_tokens(x, bsp.INT8, eps=-1.0)
    assert e.value.status == bsp.E_ARG
    with pytest.raises(TypeError):
        bsp.quantize_tokens(x, bsp.INT8, weight=np.ones(64, np.float16))
    with pytest.raises(TypeError):
        bsp.dequantize_tokens(x, torch.zeros(2, device=dev), bsp.INT8, 64)


def test_calls_from_several_threads(dev):
    x = [torch.randn(100, 512, device=dev).half() for _ in range(4)]
    want = [bsp.quantize_tokens(a, bsp.INT8) for a in x]
    got = [None] * 4
    torch.cuda.synchronize()

    def work(i):
        for _ in range(50):
            got[i] = bsp.quantize_tokens(x[i], bsp.INT8)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)


def test_calls_from_several_threads(dev):
    # each on a stream and a workspace of its own; the launch gives up the interpreter's lock
    rng = np.random.default_rng(12)
    W = rng.integers(-128, 128, (512, 11008)).astype(np.int8)
    enc = bsp.encode_int8(W, np.full(512, 1e-4, np.float32)).to_device(dev)
    X = torch.from_numpy(rng.normal(0, 1, (600, 11008)).astype(np.float16)).to(dev)
    t = bsp.quantize_tokens(X, bsp.INT8)
    want = bsp.gemm_w8a8(enc, t.codes, t.scale)
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ws = bsp.new_gemm_workspace(enc, 600, device=dev)
                for n in (600, 1, 33, 600, 257, 16):
                    q = bsp.quantize_tokens(X[:n], bsp.INT8)
                    Y = bsp.gemm_w8a8(enc, q.codes, q.scale, workspace=ws)
                    back = bsp.dequantize_tokens(q.codes, q.scale, bsp.INT8, 11008)
                    stream.synchronize()
                    if not (torch.equal(Y, want[:n]) and torch.equal(q.codes, t.codes[:n]) and torch.isfinite(back).all()):
                        wrong.append(n)
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not wrong
