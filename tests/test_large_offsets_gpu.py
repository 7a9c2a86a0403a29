"""MXFP4 products, norm and gate whose outputs pass 2^31 elements or 2^32 bytes:
the rows and columns at both ends and around the borders."""
import pytest
import torch

from mxfp8_w8a8_quantized_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def _codes(rows, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)


def _values(codes):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    grid = torch.cat([grid, -grid])
    return grid[torch.stack([codes & 15, codes >> 4], dim=-1).view(codes.shape[0], -1).long()]


# the large kernel, more rows than 2^31 / N; the few-rows kernel, a wide output
@pytest.mark.parametrize("M,K,N", [(140000, 64, 16384), (128, 32, (1 << 24) + 8), (1, 32, (1 << 25) + 8)])
def test_product(mx, M, K, N):
    """Scales of 1 and short K: products and sums are exact in binary32."""
    xq, wq = _codes(M, K, M), _codes(N, K, N + 1)
    xs = torch.full((mx.mxfp4_scale_bytes(M, K),), 127, dtype=torch.uint8, device="cuda")
    ws = torch.full((mx.mxfp4_scale_bytes(N, K),), 127, dtype=torch.uint8, device="cuda")
    y = mx.mxfp4_gemm(xq, xs, wq, ws)
    border = (1 << 31) // N
    rows = torch.tensor(sorted({r % M for r in (0, 1, 127, 128, border - 1, border, border + 1, M - 129, M - 1)}))
    cols = torch.tensor(sorted({c % N for c in (0, 127, 128, 255, 256, (1 << 23) - 1, 1 << 24, N - 129, N - 8, N - 1)}))
    want = (_values(xq[rows.cuda()]).double() @ _values(wq[cols.cuda()]).double().t()).float().bfloat16()
    assert torch.equal(y[rows.cuda()][:, cols.cuda()], want)
    assert mx.device_status() == 0


def test_norm_and_gate(mx):
    M, K = 140000, 16384                            # 2.3e9 elements; codes of 1 byte each pass 2^31
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    base = synth.activations_device(1024, K, 1, 0, "cuda")
    for i in range(0, M, 1024):
        x[i: i + 1024] = base[: min(1024, M - i)]
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    n = 1024
    for f in (lambda t: mx.rmsnorm_quantize(t, w)[:2], lambda t: mx.fp8rw_rmsnorm_quantize(t, w)[:2],
              lambda t: mx.gated_quantize(t, t), lambda t: mx.fp8rw_gated_quantize(t, t), lambda t: mx.mxfp4_quantize(t)):
        codes, scales = f(x)
        want_c, want_s = f(base)
        for i in (0, 131072 // n * n, (M - 1) // n * n):     # 131072 x 16384 = 2^31
            k = min(n, M - i)
            assert torch.equal(codes[i: i + k], want_c[:k])
        if scales.dtype == torch.float32:
            assert torch.equal(scales[131072: 132096], want_s)
        else:
            per = scales.numel() // ((M + 127) // 128) * 8   # bytes of 1024 rows
            assert torch.equal(scales[128 * per: 129 * per], want_s[:per])
        del codes, scales
