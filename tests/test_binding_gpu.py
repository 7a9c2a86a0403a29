"""Arguments that the compiled binding refuses before the library is called."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


@pytest.mark.parametrize("beyond", [1 << 32, -(1 << 32), 1 << 31, 1 << 70])
def test_integers_beyond_32_bits(mx, beyond):
    """2^32 + an activation or layout is not that activation or layout."""
    x = torch.randn(4, 64, device="cuda").bfloat16()
    w = torch.ones(64, device="cuda").bfloat16()
    for call in (lambda: mx.gated_quantize(x, x, mx.ACT_SILU + beyond),
                 lambda: mx.gated_quantize(x, x, layout=mx.SF_TCGEN05 + beyond),
                 lambda: mx.fp8rw_gated_quantize(x, x, mx.ACT_GELU_TANH + beyond),
                 lambda: mx.mxfp4_gated_quantize(x, x, mx.ACT_SILU + beyond),
                 lambda: mx.rmsnorm_quantize(x, w, layout=mx.SF_TCGEN05 + beyond)):
        with pytest.raises((ValueError, mx.MXFP8Error)):
            call()


def test_wrong_kinds(mx):
    x = torch.randn(4, 64, device="cuda").bfloat16()
    w = torch.ones(64, device="cuda").bfloat16()
    for call in (lambda: mx.gated_quantize(x, x, 2.0), lambda: mx.gated_quantize(x, x, "silu"),
                 lambda: mx.rmsnorm_quantize(x, w, "small"), lambda: mx.rmsnorm_quantize(x, w, layout=None)):
        with pytest.raises(TypeError):
            call()
