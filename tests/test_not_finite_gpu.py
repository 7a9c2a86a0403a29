"""Infinities and NaN in every quantized format: the per-channel FP8 quantizers
against the oracle's divisions, and the gated activation against the
stand-alone quantizers, which it must equal where its result is a BF16 value."""
import numpy as np
import pytest
import torch

import oracle
from helpers import bf16_bits
from mxfp8_w8a8_quantized_b200 import synth

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
FORMATS = ("mxfp8", "mxfp8_rows", "fp8rw", "nvfp4", "mxfp4")


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def _rows_with_inf(M, K, dtype):
    x = synth.activations_device(M, K, M + K, 0, "cuda").to(dtype)
    x[1, K // 2] = INF
    x[2, 3], x[2, K - 1] = -INF, INF
    x[3] = INF
    x[4, 0] = 0.0
    x[4, 1] = -INF
    return x


# staged rows, one CTA per row (16384), and the shortest
@pytest.mark.parametrize("K", [8, 520, 5120, 16384])
def test_rowwise_quantizer_rows_with_inf(mx, K):
    x = _rows_with_inf(7, K, torch.bfloat16)
    codes, scales = mx.fp8rw_quantize(x)
    rq, rs = oracle.quantize_rowwise_bf16(bf16_bits(x))
    assert np.array_equal(codes.cpu().numpy(), rq)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), rs.view(np.uint32))


@pytest.mark.parametrize("K", [8, 1024, 13824])
def test_rowwise_weight_quantizer_rows_with_inf(mx, K):
    w = _rows_with_inf(9, K, torch.float32)
    codes, scales = mx.fp8rw_quantize_weight(w)
    rq, rs = oracle.quantize_rowwise_f32(w.cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), rq)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), rs.view(np.uint32))


def _gated(mx, fmt, g, u, act, scale):
    if fmt == "mxfp8":
        return mx.gated_quantize(g, u, act)
    if fmt == "mxfp8_rows":
        return mx.gated_quantize(g, u, act, layout=mx.SF_ROWMAJOR)
    if fmt == "nvfp4":
        return mx.nvfp4_gated_quantize(g, u, scale, act)
    return getattr(mx, f"{fmt}_gated_quantize")(g, u, act)


def _alone(mx, fmt, y, scale):
    if fmt == "mxfp8":
        return mx.quantize(y)
    if fmt == "mxfp8_rows":
        return mx.quantize(y, layout=mx.SF_ROWMAJOR)
    if fmt == "nvfp4":
        return mx.nvfp4_quantize(y, scale)
    return getattr(mx, f"{fmt}_quantize")(y)


@pytest.mark.parametrize("act", ("silu", "gelu_tanh"))
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [64, 544, 5120, 16384])
def test_gate_equals_the_stand_alone_quantizer(mx, fmt, act, K):
    """A gate of 128: e^-128 is below half a step of 1 and act(128) = 128, so y
    = 128 up is the BF16 value itself, Inf where it passes the largest."""
    M = 12
    u = synth.activations_device(M, K, K, 0, "cuda")
    u[1, K // 2] = INF
    u[2, 3], u[2, K - 1] = -INF, INF
    u[3] = INF
    u[4, 7] = NAN
    u[5, 1], u[5, K - 2] = NAN, INF
    u[6, 9] = 3e38                                  # finite; 128 times it is not
    u[7] = 0.0
    u[8] = 0.0
    u[8, K // 2 + 1] = -3e38
    g = torch.full_like(u, 128.0)
    scale = torch.tensor([0.75], device="cuda")
    y = (u.float() * 128.0).to(torch.bfloat16)
    got = _gated(mx, fmt, g, u, mx.ACT_SILU if act == "silu" else mx.ACT_GELU_TANH, scale)
    want = _alone(mx, fmt, y, scale)
    assert torch.equal(got[0], want[0])
    a, b = got[1], want[1]
    if fmt == "fp8rw":
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
        s = a.cpu().numpy()
        assert np.isinf(s[[1, 2, 3, 6, 8]]).all() and np.isnan(s[[4, 5]]).all() and np.isfinite(s[[0, 7, 9, 10, 11]]).all()
        assert set((got[0][1] & 0x7F).unique().tolist()) == {0, 0x7F} and int((got[0][1] == 0x7F).sum()) == 1
    else:
        n = min(a.numel(), b.numel())
        assert torch.equal(a[:n], b[:n])


@pytest.mark.parametrize("fmt", FORMATS)
def test_infinite_gates(mx, fmt):
    """act(Inf) = Inf, act(-Inf) = NaN as the formulas have it (-Inf times 0)."""
    M, K = 5, 544
    u = synth.activations_device(M, K, 3, 0, "cuda")
    u[:, 40] = 2.0
    g = torch.full_like(u, 128.0)
    scale = torch.tensor([0.75], device="cuda")
    y = u.float() * 128.0
    g[1, 40], g[3, 40] = INF, -INF
    y[1, 40], y[3, 40] = INF, NAN
    for act in (mx.ACT_SILU, mx.ACT_GELU_TANH):
        got = _gated(mx, fmt, g, u, act, scale)
        want = _alone(mx, fmt, y.to(torch.bfloat16), scale)
        assert torch.equal(got[0], want[0])
        if fmt == "fp8rw":
            assert torch.equal(torch.nan_to_num(got[1]), torch.nan_to_num(want[1])) and bool(torch.isnan(got[1][3]))
        else:
            n = min(got[1].numel(), want[1].numel())
            assert torch.equal(got[1][:n], want[1][:n])
