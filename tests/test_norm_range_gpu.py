"""The RMS norm over the whole range of BF16 and to the precision its kernel
states, in every format, against the 64-bit form.

Squares are formed and summed in binary64 (errors of 2^-50), and with a BF16
weight the product h w has at most 16 bits, so it is exact in binary32 while it
is normal.  rstd is applied as a pair of binary32 values, which hold it to
2^-48; what is left is the rounding of y, half a step (u = 2^-24), and the
lower product's own, 2^-24 u.  So y is within 1.01 u of the formula; a row's
scale of per-channel FP8 is RN(RN(y) / 448), 2.01 u.  Where the root mean
square passes 2^100, the pair's lower part is subnormal or zero (u more), from
2^126 on the upper one as well, which has 2^-150 / 2^-128 = 4 u at the top:
4 u + u, 5.01 u."""
import numpy as np
import pytest
import torch

import fused_ref as ref
from helpers import unswizzle
from mxfp8_w8a8_quantized_b200 import synth

pytestmark = pytest.mark.gpu
EPS = 1e-6
D = 1.01 * ref.U
FORMATS = ("mxfp8", "mxfp8_rows", "fp8rw", "nvfp4", "mxfp4")
FAR = 5.01 * ref.U
# y below 2^-126 is rounded to 2^-150, t rl as well, and t, too, times rstd (at
# most 2^10 with this eps): 2^-139 covers them
TINY = 2.0 ** -139


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def _run(mx, fmt, x, w, eps=EPS, **k):
    if fmt == "mxfp8":
        return mx.rmsnorm_quantize(x, w, eps, **k)
    if fmt == "mxfp8_rows":
        return mx.rmsnorm_quantize(x, w, eps, layout=mx.SF_ROWMAJOR, **k)
    if fmt == "nvfp4":
        return mx.nvfp4_rmsnorm_quantize(x, w, torch.tensor([37.5], device="cuda"), eps, **k)
    return getattr(mx, f"{fmt}_rmsnorm_quantize")(x, w, eps, **k)


def _check(fmt, codes, scales, y, extra=0.0, what="", d=D):
    M, K = y.shape
    q, s = codes.cpu().numpy(), scales.cpu().numpy()
    if fmt == "fp8rw":
        return ref.check_rowwise(ref.decode_e4m3(q), s, y, d, extra, what)
    if fmt == "mxfp8_rows":
        return ref.check_mx(ref.decode_e4m3(q), s.reshape(M, K // 32), y, d, extra, what=what, typical=False)
    rows = unswizzle(s, M, K, 16 if fmt == "nvfp4" else 32)
    if fmt == "mxfp8":
        ref.check_mx(ref.decode_e4m3(q), rows, y, d, extra, what=what, typical=False)
    elif fmt == "mxfp4":
        ref.check_mx(ref.unpack_e2m1(q), rows, y, d, extra, emax=2, grid=ref.E2M1, what=what, typical=False)
    else:
        ref.check_nvfp4(q, rows, 37.5, y, d, extra, what)


def _weight(K, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(dtype)


def _formula(h, w, eps=EPS):
    return ref.rmsnorm(h, w, float(np.float32(eps)))


# one K per variant: a warp's row, 128 threads with few and many chunks, 256, 512
@pytest.mark.parametrize("K", [1024, 2048, 5120, 8192, 16384])
def test_row_scale_is_the_formulas_to_two_roundings(mx, K):
    """Large elements first, then many whose square is just below half a step
    of the running sum's (1): a sum in binary32 loses every one of them."""
    M = 16
    x = torch.full((M, K), 1.9921875 * 2.0 ** -13, dtype=torch.bfloat16, device="cuda")
    lead = torch.arange(K, device="cuda")
    for r in range(M):
        n = K // (r + 1) // 8 * 8                   # 1.0 in the first n, two of eight
        x[r, (lead < n) & (lead % 8 < 2)] = 1.0
    x[M - 1] = 1.9921875 * 2.0 ** -13
    w = _weight(K, K)
    y = _formula(x, w)
    s = mx.fp8rw_rmsnorm_quantize(x, w, EPS)[1].double().cpu().numpy()
    want = np.abs(y).max(-1) / 448.0
    off = np.abs(s / want - 1.0) / ref.U
    assert off.max() <= 2.01, f"K = {K}: {off.max():.2f} half steps off, row {off.argmax()}"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(600, 1024), (512, 5120), (64, 16384)])
def test_codes_are_the_formulas_to_one_rounding(mx, fmt, M, K):
    x = synth.activations_device(M, K, M + K, 0, "cuda")
    r = synth.activations_device(M, K, M + K, 1, "cuda")
    x[:, 7::64] *= 30.0
    w = _weight(K, M)
    codes, scales, h = _run(mx, fmt, x, w, residual=r)
    assert torch.equal(h, (x.double() + r.double()).to(torch.bfloat16))
    _check(fmt, codes, scales, _formula(h, w), what=f"{fmt} {M}x{K}")


@pytest.mark.parametrize("dtype,d", [(torch.float16, D), (torch.float32, 2.01 * ref.U)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_codes_with_other_weight_types(mx, fmt, dtype, d):
    """An FP16 weight's product has 19 bits; an FP32 one's is rounded once more."""
    M, K = 400, 5120
    x = synth.activations_device(M, K, 31, 0, "cuda")
    w = _weight(K, 32, dtype)
    codes, scales, _ = _run(mx, fmt, x, w)
    _check(fmt, codes, scales, _formula(x, w), what=f"{fmt} {dtype}", d=d)


BIG = 1.7e38        # times the largest weight here, 1.9, still a binary32


def _bound(h):
    """Relative bound of each row's y."""
    rms = h.double().square().mean(-1, keepdim=True).sqrt().cpu().numpy()
    return np.where(rms > 2.0 ** 100, FAR, D)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [96, 2048, 5120, 8192, 16384])
def test_rows_of_any_finite_size(mx, fmt, K):
    """The squares of these rows pass binary32 in one direction or the other."""
    sizes = (1e15, 1e18, 1.8e19, 1.9e19, 1e20, 1e25, 1e30, 1e36, 1e38, 1e-15, 1e-19, 1e-25)
    M = len(sizes) + 6
    x = synth.activations_device(M, K, K, 0, "cuda").float().clamp_(-60.0, 60.0)
    x = x * (torch.tensor(sizes + (1.0,) * 6, device="cuda") / 64.0)[:, None]
    x = x.to(torch.bfloat16)
    x[-6] = 1e30
    x[-5] = BIG
    x[-4, ::2], x[-4, 1::2] = -BIG, BIG
    x[-3, K - 1] = 1e30                            # one element far above the rest
    x[-2, 3] = -BIG
    x[-1] = 0.0
    x[-1, 5] = 1.9e19
    assert torch.isfinite(x).all()
    w = _weight(K, 3)
    w.clamp_(max=1.9)
    w[3], w[K - 1] = 1.9, 1.7
    codes, scales, _ = _run(mx, fmt, x, w)
    y = _formula(x, w)
    _check(fmt, codes, scales, y, TINY, f"{fmt} K = {K}", _bound(x))
    # the rows around them keep their values
    for r in (0, M - 3):
        a = _run(mx, fmt, x[r:r + 1], w)
        assert torch.equal(a[0], codes[r:r + 1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_residual_stream_of_any_size_and_in_place(mx, fmt):
    M, K = 9, 5120
    x = synth.activations_device(M, K, 5, 0, "cuda")
    r = synth.activations_device(M, K, 5, 1, "cuda")
    x[2] *= 1e25
    r[3] *= 1e36
    x[4], r[4] = 8e37, 8e37
    w = _weight(K, 4)
    want = (x.double() + r.double()).to(torch.bfloat16)
    codes, scales, h = _run(mx, fmt, x, w, residual=r, residual_out=r)
    assert h is r and torch.equal(h, want) and torch.isfinite(h).all()
    _check(fmt, codes, scales, _formula(h, w), TINY, fmt, _bound(h))


def test_squares_below_binary32(mx):
    """With the smallest eps a row's squares decide although binary32 does not
    hold them."""
    K, eps = 1056, 1.5e-45
    x = (synth.activations_device(6, K, 6, 0, "cuda").float() *
         torch.tensor([1e-22, 1e-23, 1e-21, 1e-25, 1e-30, 1.0], device="cuda")[:, None]).to(torch.bfloat16)
    w = _weight(K, 5)
    y = _formula(x, w, eps)
    s = mx.fp8rw_rmsnorm_quantize(x, w, eps)[1].double().cpu().numpy()
    assert np.all(np.abs(s / (np.abs(y).max(-1) / 448.0) - 1.0) <= 2.01 * ref.U)


@pytest.mark.parametrize("fmt", FORMATS)
def test_inf_and_nan_stay_in_their_rows(mx, fmt):
    """Inf: the row's finite elements come out as zeros whatever their size, its
    own block as NaN; per row (one scale) the whole row."""
    M, K = 6, 5120
    x = synth.activations_device(M, K, 7, 0, "cuda")
    w = _weight(K, 6)
    want = _run(mx, fmt, x, w)
    x[1, 100], x[1, 40], x[3, 4] = float("inf"), BIG, float("nan")
    codes, scales, _ = _run(mx, fmt, x, w)
    keep = [0, 2, 4, 5]
    assert torch.equal(codes[keep], want[0][keep])
    q = codes.cpu().numpy()
    if fmt == "fp8rw":
        s = scales.cpu().numpy()
        assert np.isnan(s[[1, 3]]).all() and np.array_equal(s[keep], want[1].cpu().numpy()[keep])
        assert np.all(q[[1, 3]] == 0x7F)
        return
    if fmt == "nvfp4":
        return
    s = scales.cpu().numpy()
    s = s.reshape(M, -1) if fmt == "mxfp8_rows" else unswizzle(s, M, K)
    assert np.all(s[3] == 255) and s[1, 3] == 255
    assert not s[1, :3].any() and not s[1, 4:].any()
    fp4 = fmt == "mxfp4"
    v = ref.unpack_e2m1(q) if fp4 else ref.decode_e4m3(q)
    assert not v[1, :96].any() and not v[1, 128:].any()


def test_product_beyond_binary32_is_inf(mx):
    """h w past 3.4e38 comes out as Inf in its block; the others keep theirs."""
    K = 1056
    x = torch.full((2, K), 3e38, dtype=torch.bfloat16, device="cuda")
    w = torch.full((K,), 1.0, dtype=torch.bfloat16, device="cuda")
    w[70] = 2.0
    codes, scales, _ = mx.rmsnorm_quantize(x, w, EPS)
    s, v = unswizzle(scales.cpu().numpy(), 2, K), ref.decode_e4m3(codes.cpu().numpy())
    assert np.all(s[:, 2] == 255) and np.all(np.delete(s, 2, axis=1) == 127 - 8)
    assert np.all(np.delete(v.reshape(2, -1, 32), 2, axis=1) == 256.0)
