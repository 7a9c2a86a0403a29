"""The RMS norm, the gated activation and the MXFP4 layer without a GPU: the
C-ABI and the binding refuse bad calls before anything is launched, and the
64-bit reference forms the GPU tests compare with are pinned to the formats'
definitions."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import fused_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # a 16-byte aligned, never dereferenced address
ARG, ALIGN, SHAPE = 1, 2, 3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import build
    build.build()
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def test_mxfp4_header_and_binding_agree(mx):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxfp4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(mxfp4_[a-z0-9_]+)\s*\(", text))
    assert names == set(mx.MXFP4_EXPORTS)
    for n in names:
        assert hasattr(mx._lib, n)


# ----------------------------------------------------------------- C-ABI
def _norm(mx, fn, x=FAKE, ldx=64, r=None, ldr=0, h=None, ldh=0, w=FAKE, dt=0, eps=1e-6, M=4, K=64, tail=None):
    tails = {"mxfp8": (FAKE, FAKE, 1, None), "fp8rw": (FAKE, FAKE, None), "nvfp4": (FAKE, FAKE, FAKE, None),
             "mxfp4": (FAKE, FAKE, None)}
    return getattr(mx._lib, f"{fn}_rmsnorm_quantize")(x, ldx, r, ldr, h, ldh, w, dt, eps, M, K, *(tail or tails[fn]))


@pytest.mark.parametrize("fn", ["mxfp8", "fp8rw", "nvfp4", "mxfp4"])
def test_norm_refuses_before_launch(mx, fn):
    n = lambda **k: _norm(mx, fn, **k)
    assert n(M=0) == 0                                       # empty: no-op
    assert n(M=0, x=None, w=None) == 0
    assert n(x=None) == ARG and n(w=None) == ARG
    assert n(M=-1) == ARG and n(K=0) == ARG
    assert n(ldx=32) == ARG                                  # row stride < K
    assert n(dt=3) == ARG and n(dt=-1) == ARG
    for eps in (0.0, -1e-6, NAN, INF, 1e-60):                # 1e-60 is 0 in binary32
        assert n(eps=eps) == ARG
    assert n(K=68, ldx=72) == SHAPE                          # K of no format
    assert n(K=16416, ldx=16416) == SHAPE                    # longer than a row may be
    assert n(M=(1 << 30) + 1) == SHAPE
    assert n(x=FAKE + 2) == ALIGN and n(ldx=68) == ALIGN and n(w=FAKE + 8) == ALIGN
    # residual: its output is needed, in place only with one stride
    assert n(r=FAKE, ldr=64) == ARG
    assert n(r=FAKE, ldr=32, h=FAKE + 4096, ldh=64) == ARG
    assert n(r=FAKE, ldr=64, h=FAKE + 4096, ldh=32) == ARG
    assert n(r=FAKE + 4096, ldr=64, h=FAKE, ldh=128) == ARG
    assert n(x=FAKE + 4096, r=FAKE, ldr=64, h=FAKE, ldh=128) == ARG
    assert n(r=FAKE + 8, ldr=64, h=FAKE + 4096, ldh=64) == ALIGN
    assert n(r=FAKE, ldr=64, h=FAKE + 4100, ldh=64) == ALIGN


def test_norm_refuses_bad_outputs(mx):
    assert _norm(mx, "mxfp8", tail=(None, FAKE, 1, None)) == ARG
    assert _norm(mx, "mxfp8", tail=(FAKE, None, 1, None)) == ARG
    assert _norm(mx, "mxfp8", tail=(FAKE, FAKE, 2, None)) == ARG             # layout
    assert _norm(mx, "mxfp8", tail=(FAKE + 4, FAKE, 1, None)) == ALIGN
    assert _norm(mx, "fp8rw", tail=(FAKE, FAKE + 2, None)) == ALIGN
    assert _norm(mx, "nvfp4", tail=(None, FAKE, FAKE, None)) == ARG          # global scale
    assert _norm(mx, "nvfp4", tail=(FAKE + 2, FAKE, FAKE, None)) == ALIGN
    assert _norm(mx, "mxfp4", K=48, ldx=48) == SHAPE
    assert _norm(mx, "mxfp8", K=48, ldx=48) == SHAPE
    assert _norm(mx, "nvfp4", K=24, ldx=24) == SHAPE


def _gated(mx, fn, g=FAKE, ldg=64, u=FAKE, ldu=64, act=2, M=4, K=64, tail=None):
    tails = {"mxfp8": (FAKE, FAKE, 1, None), "fp8rw": (FAKE, FAKE, None), "nvfp4": (FAKE, FAKE, FAKE, None),
             "mxfp4": (FAKE, FAKE, None)}
    return getattr(mx._lib, f"{fn}_gated_quantize")(g, ldg, u, ldu, act, M, K, *(tail or tails[fn]))


@pytest.mark.parametrize("fn", ["mxfp8", "fp8rw", "nvfp4", "mxfp4"])
def test_gated_refuses_before_launch(mx, fn):
    n = lambda **k: _gated(mx, fn, **k)
    assert n(M=0) == 0 and n(M=0, g=None) == 0
    assert n(act=0) == ARG and n(act=3) == ARG               # a gate has an activation
    assert n(g=None) == ARG and n(u=None) == ARG
    assert n(M=-1) == ARG and n(K=0) == ARG
    assert n(ldg=32) == ARG and n(ldu=32) == ARG
    assert n(K=68, ldg=72, ldu=72) == SHAPE
    big = 16392 if fn == "fp8rw" else (1 << 20) + 32
    assert n(K=big, ldg=big, ldu=big) == SHAPE
    assert n(g=FAKE + 2) == ALIGN and n(u=FAKE + 8) == ALIGN and n(ldg=68) == ALIGN and n(ldu=68) == ALIGN


def test_mxfp4_refuses_before_launch(mx):
    L = mx._lib
    assert L.mxfp4_scale_bytes(1, 32) == 512 and L.mxfp4_scale_bytes(129, 160) == 2 * 2 * 512
    assert L.mxfp4_scale_bytes(10, 48) == 0 and L.mxfp4_scale_bytes(-1, 32) == 0
    assert L.mxfp4_quantize_bf16(None, 4, 64, 64, FAKE, FAKE, None) == ARG
    assert L.mxfp4_quantize_bf16(FAKE, 4, 64, 32, FAKE, FAKE, None) == ARG
    assert L.mxfp4_quantize_bf16(FAKE, 4, 48, 48, FAKE, FAKE, None) == SHAPE
    assert L.mxfp4_quantize_bf16(FAKE, 4, 64, 68, FAKE, FAKE, None) == ALIGN
    assert L.mxfp4_quantize_bf16(FAKE, 4, 64, 64, FAKE + 4, FAKE, None) == ALIGN
    assert L.mxfp4_quantize_bf16(FAKE, 0, 64, 64, FAKE, FAKE, None) == 0
    assert L.mxfp4_quantize_weight_f32(FAKE, 4, 40, FAKE, FAKE, None) == SHAPE
    assert L.mxfp4_quantize_weight_f32(FAKE + 4, 4, 64, FAKE, FAKE, None) == ALIGN
    for M in (4, 4000):                                      # the few-rows kernel and the other
        assert L.mxfp4_gemm(FAKE, FAKE, M, 48, FAKE, FAKE, 16, None, FAKE, None) == SHAPE
        assert L.mxfp4_gemm(FAKE, FAKE, M, 64, FAKE, FAKE, 12, None, FAKE, None) == SHAPE
        assert L.mxfp4_gemm(FAKE, FAKE + 4, M, 64, FAKE, FAKE, 16, None, FAKE, None) == ALIGN
        assert L.mxfp4_gemm(FAKE, FAKE, M, 64, FAKE, FAKE, 16, FAKE + 2, FAKE, None) == ALIGN
        assert L.mxfp4_gemm(FAKE, FAKE, M, 64, FAKE, None, 16, None, FAKE, None) == ARG
        assert L.mxfp4_gemm(FAKE, FAKE, M, 64, FAKE, FAKE, 0, None, FAKE, None) == ARG
    assert L.mxfp4_gemm(FAKE, FAKE, 0, 64, FAKE, FAKE, 16, None, FAKE, None) == 0
    need = L.mxfp4_linear_workspace_bytes(4, 160)
    assert need == 512 + 2 * 512
    assert L.mxfp4_linear(FAKE, 4, 160, FAKE, FAKE, 16, None, FAKE, FAKE, need - 1, None) == ARG
    assert L.mxfp4_linear(FAKE, 4, 160, FAKE, FAKE, 16, None, FAKE, FAKE + 16, need, None) == ALIGN
    assert L.mxfp4_linear(FAKE, 4, 48, FAKE, FAKE, 16, None, FAKE, FAKE, need, None) == SHAPE
    assert L.mxfp4_linear(FAKE, 4, 160, FAKE, FAKE, 12, None, FAKE, FAKE, need, None) == SHAPE
    assert L.mxfp4_linear(FAKE, 4, 160, FAKE, FAKE + 4, 16, None, FAKE, FAKE, need, None) == ALIGN
    assert L.mxfp4_linear(FAKE, 4, 160, FAKE, FAKE, 16, None, None, FAKE, need, None) == ARG


def test_binding_refuses_host_tensors(mx):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    f32 = lambda *s: torch.zeros(*s, dtype=torch.float32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    calls = [
        lambda: mx.mxfp4_quantize(bf(4, 64)),
        lambda: mx.mxfp4_quantize_weight(f32(8, 64)),
        lambda: mx.mxfp4_gemm(u8(4, 32), u8(512), u8(8, 32), u8(512)),
        lambda: mx.mxfp4_linear(bf(4, 64), u8(8, 32), u8(512)),
        lambda: mx.rmsnorm_quantize(bf(4, 64), bf(64)),
        lambda: mx.fp8rw_rmsnorm_quantize(bf(4, 64), bf(64)),
        lambda: mx.nvfp4_rmsnorm_quantize(bf(4, 64), bf(64), f32(1)),
        lambda: mx.mxfp4_rmsnorm_quantize(bf(4, 64), bf(64)),
        lambda: mx.gated_quantize(bf(4, 64), bf(4, 64)),
        lambda: mx.fp8rw_gated_quantize(bf(4, 64), bf(4, 64)),
        lambda: mx.nvfp4_gated_quantize(bf(4, 64), bf(4, 64), f32(1)),
        lambda: mx.mxfp4_gated_quantize(bf(4, 64), bf(4, 64)),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_selftest_of_the_few_rows_wait_is_known(mx):
    assert mx._lib.mxfp8_selftest_wait_timeout(mx.SELFTEST_MXFP4_FEW_ROWS, 0, None) == ARG   # no limit
    assert mx._lib.mxfp8_selftest_wait_timeout(5, 1000000, None) == ARG


# ------------------------------------------------- pins of the references
def test_reference_e4m3_is_torchs():
    assert len(ref.E4M3) == 127
    assert np.array_equal(ref.E4M3, ref.decode_e4m3(np.arange(127, dtype=np.uint8)))
    v = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.exp2(np.arange(20000) % 20 - 12)
    v = np.concatenate([v, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2, [0.0, -0.0, 448.0, 464.0, 1e6, 2.0 ** -10]])
    t = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.round_grid(v, ref.E4M3), t)


def test_reference_e2m1_by_hand():
    v = np.array([0.25, 0.250001, 0.75, 0.749999, 1.25, 1.75, 2.5, 2.500001, 3.5, 3.499999, 5.0, 5.000001, 7.0, -0.1, -2.6])
    w = np.array([0.0, 0.5, 1.0, 0.5, 1.0, 2.0, 2.0, 3.0, 4.0, 3.0, 4.0, 6.0, 6.0, -0.0, -3.0])
    got = ref.round_grid(v, ref.E2M1)
    assert np.array_equal(got, w) and np.array_equal(np.signbit(got), np.signbit(w))


def test_reference_mxfp4_block_by_hand():
    x = np.zeros((1, 64))
    x[0, :4] = [6.0, -3.0, 0.25, 7.9]            # amax 7.9: e = 2 - 2 = 0
    x[0, 32] = -0.4                              # e = -2 - 2 = -4: 0.4 * 16 = 6.4 -> 6
    q, s = ref.mxfp4_quantize(x)
    assert s.tolist() == [[127, 123]]
    assert q[0, :2].tolist() == [7 | (13 << 4), 0 | (7 << 4)] and q[0, 16] == 15
    assert ref.mxfp4_values(q, s)[0, 32] == -0.375
    q, s = ref.mxfp4_quantize(np.full((1, 32), np.inf))
    assert s[0, 0] == 255 and np.all(q == 0x77)
    assert np.all(ref.mxfp4_quantize(np.zeros((1, 32)))[1] == 0)


def test_reference_gated_is_torchs():
    g = torch.linspace(-30, 30, 2001, dtype=torch.float64)
    one = torch.ones_like(g)
    y, _, _ = ref.gated(g, one, "silu")
    assert np.allclose(y, torch.nn.functional.silu(g).numpy(), rtol=1e-12, atol=0)
    y, _, _ = ref.gated(g, one, "gelu_tanh")
    t = torch.nn.functional.gelu(g, approximate="tanh").numpy()
    assert np.allclose(y, t, rtol=1e-9, atol=1e-15)    # torch's form cancels far below zero


def test_checks_catch_a_wrong_code():
    """The interval checks refuse codes, scales and rows that are off by one."""
    rng = np.random.default_rng(1)
    y = rng.standard_normal((4, 64))
    e = ref.mx_exponent(np.abs(y).reshape(4, 2, 32).max(-1), 8)
    v = ref.round_grid(y * np.repeat(np.ldexp(1.0, -e), 32, axis=1), ref.E4M3)
    sb = (e + 127).astype(np.uint8)
    ref.check_mx(v, sb, y, ref.NORM_D)
    w = v.copy()
    w[1, 3] *= 1.125
    with pytest.raises(AssertionError):
        ref.check_mx(w, sb, y, ref.NORM_D)
    with pytest.raises(AssertionError):
        ref.check_mx(v, sb + 1, y, ref.NORM_D)
    s = np.abs(y).max(-1) / 448.0
    ref.check_rowwise(ref.round_grid(y / s[:, None], ref.E4M3), s, y, ref.NORM_D)
    with pytest.raises(AssertionError):
        ref.check_rowwise(ref.round_grid(y / s[:, None], ref.E4M3), s * 1.0001, y, ref.NORM_D)
