"""A launch that waits for room in the queue of launches does not hold up the
program's other Python threads."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
HOLD = 1.0          # seconds, about, for which the GPU is busy and the queue fills up


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def test_other_threads_run_while_a_launch_waits(mx):
    x = torch.randn(4, 512, device="cuda").bfloat16()
    w = torch.ones(512, device="cuda").bfloat16()
    wq, ws = mx.mxfp4_quantize_weight(torch.randn(64, 512, device="cuda"))
    q, s, h = mx.mxfp4_rmsnorm_quantize(x, w)
    y = mx.mxfp4_gemm(q, s, wq, ws)
    wk = torch.empty(mx.mxfp4_linear_workspace_bytes(4, 512), dtype=torch.uint8, device="cuda")
    codes, scales = mx.fp8rw_gated_quantize(x, x)
    calls = {
        "norm": lambda: mx.mxfp4_rmsnorm_quantize(x, w, codes=q, scales=s),
        "gate": lambda: mx.fp8rw_gated_quantize(x, x, codes=codes, scales=scales),
        "quantize": lambda: mx.mxfp4_quantize(x, codes=q, scales=s),
        "gemm": lambda: mx.mxfp4_gemm(q, s, wq, ws, out=y),
        "linear": lambda: mx.mxfp4_linear(x, wq, ws, out=y, workspace=wk),
    }
    # cycles that keep the GPU busy for HOLD
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    torch.cuda._sleep(10_000_000)
    b.record()
    torch.cuda.synchronize()
    cycles = int(10_000_000 * HOLD * 1e3 / a.elapsed_time(b))
    for name, call in calls.items():
        gaps, longest, failed = [], [], []

        def launches():
            try:
                for _ in range(3000):                # more than the queue holds (1024)
                    t = time.perf_counter()
                    call()
                    longest.append(time.perf_counter() - t)
            except Exception as e:
                failed.append(e)

        torch.cuda._sleep(cycles)
        thread = threading.Thread(target=launches)
        thread.start()
        last = time.perf_counter()
        while thread.is_alive():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now
        thread.join()
        torch.cuda.synchronize()
        assert not failed, failed
        # the queue was full, and the other thread did not wait for the launch that
        # waited for room (with the lock held, its gap is the whole of that wait)
        assert max(longest) > 0.1, f"{name}: no launch waited ({max(longest):.3f} s)"
        assert max(gaps) < max(longest) / 2, f"{name}: the other thread stood still for {max(gaps):.3f} s"
