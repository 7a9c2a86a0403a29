"""The first calls of a process made by several host threads at once: what the
library learns about the device on first use (resident clusters, attributes)
is filled by whichever thread comes first, and every thread's result has the
bits of later calls.  And a product as the first thing a host thread calls."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from mxfp8_w8a8_quantized_b200 import synth

pytestmark = pytest.mark.gpu

CODE = """
import ctypes, sys, threading
import torch
from mxfp8_w8a8_quantized_b200 import mxfp8 as mx, synth
M, K, N = (int(a) for a in sys.argv[1:4])
P = lambda t: ctypes.c_void_p(t.data_ptr())
THREADS = 8
# operands from elementary operations, so that no launch of the library comes first
torch.manual_seed(M)
def operand(rows):
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda")
    return codes, torch.full((mx.mxfp4_scale_bytes(rows, K),), 122, dtype=torch.uint8, device="cuda")
x, w = operand(M), operand(N)
gate = torch.randn(M, 16384, device="cuda").bfloat16()
ys = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(THREADS + 1)]
qs = [(torch.empty(M, 16384, dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda")) for _ in ys]
streams = [torch.cuda.Stream() for _ in ys]
torch.cuda.synchronize()
start, bad = threading.Barrier(THREADS), []
def work(i):
    st = ctypes.c_void_p(streams[i].cuda_stream)
    torch.cuda.set_device(0)
    if i < THREADS:
        start.wait()
    a = mx._lib.mxfp4_gemm(P(x[0]), P(x[1]), M, K, P(w[0]), P(w[1]), N, None, P(ys[i]), st)
    b = mx._lib.fp8rw_gated_quantize(P(gate), 16384, P(gate), 16384, 2, M, 16384, P(qs[i][0]), P(qs[i][1]), st)
    if a or b:
        bad.append((i, a, b))
ts = [threading.Thread(target=work, args=(i,)) for i in range(THREADS)]
[t.start() for t in ts]
[t.join() for t in ts]
torch.cuda.synchronize()
work(THREADS)
torch.cuda.synchronize()
assert not bad, bad
for y, q in zip(ys[:-1], qs):
    assert torch.equal(y.view(torch.int16), ys[-1].view(torch.int16))
    assert torch.equal(q[0], qs[-1][0]) and torch.equal(q[1], qs[-1][1])
assert mx.device_status() == 0
"""


# the few-rows kernel at each of its row sizes (K split over a cluster), the large one
@pytest.mark.parametrize("M,K,N", [(1, 13824, 264), (30, 5120, 1000), (60, 5120, 1000), (128, 13824, 520), (2600, 512, 1032)])
def test_first_calls_from_several_threads(M, K, N):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE, str(M), str(K), str(N)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


@pytest.mark.parametrize("fmt", ["mxfp8", "fp8rw", "nvfp4", "mxfp4 few rows", "mxfp4 large", "mxfp4 linear"])
def test_product_is_the_first_call_of_a_thread(mx, fmt):
    """A new thread has no CUDA context until the runtime needs one."""
    M, K, N = (2600 if fmt == "mxfp4 large" else 40), 512, 1032
    x, w = synth.activations_device(M, K, 1, 0, "cuda"), synth.weights_device(N, K, 2, 0, "cuda")
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    if fmt == "mxfp8":
        a, b = mx.quantize(x), mx.quantize_weight(w)
        call = lambda: mx.gemm_prequant(*a, *b, out=out)
    elif fmt == "fp8rw":
        a, b = mx.fp8rw_quantize(x), mx.fp8rw_quantize_weight(w)
        call = lambda: mx.fp8rw_gemm(*a, *b, out=out)
    elif fmt == "nvfp4":
        one = torch.ones(1, device="cuda")
        a, b = mx.nvfp4_quantize(x, one), mx.nvfp4_quantize_weight(w, one)
        call = lambda: mx.nvfp4_gemm(*a, *b, one, one, out=out)
    elif fmt == "mxfp4 linear":
        b = mx.mxfp4_quantize_weight(w)
        call = lambda: mx.mxfp4_linear(x, *b, out=out)
    else:
        a, b = mx.mxfp4_quantize(x), mx.mxfp4_quantize_weight(w)
        call = lambda: mx.mxfp4_gemm(*a, *b, out=out)
    want = call().clone()
    torch.cuda.synchronize()
    out.fill_(-7.0)
    failed = []

    def work():
        try:
            call()
            torch.cuda.current_stream().synchronize()
        except Exception as e:
            failed.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed
    assert torch.equal(out, want)
