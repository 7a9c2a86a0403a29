"""Kernels that start while the one ahead still runs read what it wrote: the
large MXFP4 GEMM behind kernels that rewrite its bias, operands and output in
place, with nothing waited for between, against the same steps each waited for."""
import pytest
import torch

from mxfp8_w8a8_quantized_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def _weight(mx, N, K, seed, index=0):
    return mx.mxfp4_quantize_weight(synth.weights_device(N, K, seed, index, "cuda"))


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# more 128 x 128 tiles than SMs: the large kernel; and one of each smaller size
@pytest.mark.parametrize("M,K,N", [(1500, 288, 2056), (2300, 544, 1544), (4, 544, 1544), (260, 544, 1544)])
def test_bias_written_by_the_kernel_ahead(mx, M, K, N):
    """A product's row, its BF16 bits taken as FP16 ones, is the bias of the
    layer right behind it, in one buffer for all of them."""
    E = 256
    assert (M <= 260) == ((M + 127) // 128 * ((N + 127) // 128) <= _sms())
    x = synth.activations_device(M, K, 1, 0, "cuda")
    wq, ws = _weight(mx, N, K, 2)
    eq, es = _weight(mx, N, E, 3)
    emb = [synth.activations_device(1, E, 4 + i, 0, "cuda") for i in range(8)]
    row = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    bias = row.view(torch.float16)[0]
    xq, xs = mx.mxfp4_quantize(x)

    def run(pause):
        got = []
        for e in emb:
            mx.mxfp4_linear(e, eq, es, out=row)
            pause()
            got.append(mx.mxfp4_gemm(xq, xs, wq, ws, bias))
            pause()
        return got

    want = run(torch.cuda.synchronize)
    assert not torch.equal(want[0], want[1])
    for _ in range(10):
        got = run(lambda: None)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert mx.device_status() == 0


@pytest.mark.parametrize("M,K,N", [(1500, 512, 2056), (2, 512, 2056)])
def test_operands_written_by_the_kernel_ahead(mx, M, K, N):
    """Codes, scales and weights quantized into the same buffers right ahead of
    the product."""
    ws_f32 = [synth.weights_device(N, K, 11, i, "cuda") for i in range(3)]
    xs_bf = [synth.activations_device(M, K, 12, i, "cuda") for i in range(3)]
    b = synth.bias_device(N, 13, 0, "cuda")
    wq, ws = _weight(mx, N, K, 0)
    xq, xs = mx.mxfp4_quantize(xs_bf[0])
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")

    def run(pause):
        got = []
        for i in range(9):
            c, s = mx.mxfp4_quantize_weight(ws_f32[i % 3])
            pause()
            wq.copy_(c)
            ws.copy_(s)
            pause()
            mx.mxfp4_quantize(xs_bf[(i + i // 3) % 3], codes=xq, scales=xs)
            pause()
            mx.mxfp4_gemm(xq, xs, wq, ws, b, out=out)
            pause()
            got.append(out.clone())
            pause()
        return got

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        got = run(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))


@pytest.mark.parametrize("M", [1500, 2300])
def test_layers_over_the_same_buffers_in_the_large_kernel(mx, M):
    """Rows, codes and outputs rewritten in place layer after layer, in sizes
    that the large kernel takes."""
    K, N = 1568, 1056                              # a width that ends inside a scale atom
    x, r = synth.activations_device(M, K, 20, 0, "cuda"), synth.activations_device(M, K, 20, 1, "cuda")
    w = (1.0 + 0.2 * torch.randn(K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")).bfloat16()
    layers = [(_weight(mx, 2 * N, K, 21, i), _weight(mx, K, N, 22, i)) for i in range(4)]
    assert (M + 127) // 128 * ((K + 127) // 128) > _sms()

    def run(pause):
        y, h = x.clone(), r.clone()
        gu = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
        for up, down in layers:
            q, s, _ = mx.mxfp4_rmsnorm_quantize(y, w, residual=h, residual_out=h)
            pause()
            mx.mxfp4_gemm(q, s, *up, out=gu)
            pause()
            a, t = mx.mxfp4_gated_quantize(gu[:, :N], gu[:, N:], mx.ACT_SILU)
            pause()
            mx.mxfp4_gemm(a, t, *down, out=y)
            pause()
            mx.mxfp4_linear(y, *up, out=gu)
            pause()
            y[:, :N].add_(gu[:, :N])
            pause()
        return y, h

    want = run(torch.cuda.synchronize)
    assert torch.isfinite(want[0]).all()
    for _ in range(10):
        got = run(lambda: None)
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert mx.device_status() == 0


def test_library_products_between_the_layers(mx):
    """PyTorch's products on the same stream, ahead of and behind the layers of
    each size."""
    K = N = 1024
    layers = [_weight(mx, N, K, 30, i) for i in range(3)]
    dense = (torch.randn(N, K, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") / 32).bfloat16()

    def run(M, pause):
        y = synth.activations_device(M, K, 31, 0, "cuda", outliers=False)
        for wq, ws in layers:
            y = y @ dense.t()
            pause()
            y = mx.mxfp4_linear(y, wq, ws)
            pause()
            y = y @ dense.t()
            pause()
            q, s = mx.mxfp4_quantize(y)
            pause()
            y = mx.mxfp4_gemm(q, s, wq, ws)
            pause()
        return y

    for M in (1, 20, 100, 300, 2600):
        want = run(M, torch.cuda.synchronize)
        for _ in range(5):
            got = run(M, lambda: None)
            torch.cuda.synchronize()
            assert torch.equal(want, got)
    assert mx.device_status() == 0
