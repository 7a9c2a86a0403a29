"""Plain 64-bit forms of the RMS norm, the gated activations and MXFP4, and
the check of a kernel's codes and scales against them.

The formats are built here from their definitions, apart from the library and
from the oracle.  A kernel computes a value y in binary32 with a relative
error of at most d (derived per operator, below) before it quantizes, and
quantization is monotone, so a code is right exactly when it lies between the
codes of y (1 - d) and y (1 + d); the same holds for a block's scale and its
largest magnitude.  u = 2^-24 is half a step of binary32."""
import numpy as np
import torch

U = 2.0 ** -24

# norm: h w (u), times rstd (u).  The sum of squares is a sum of positive
# terms through at most 32 fused steps per thread (16 pairs, two lanes) + 1 +
# 5 shuffles + 7 warps = 45 additions, then / K and + eps: 47 u, halved by the
# square root, + u for its rounding; 27 u in all.
NORM_D = 32 * U
# gated: hardware exponential 2^-22 and reciprocal 2^-23 (both relative), up to
# 10 more roundings (8 ulp with the margin): below 2^-20.
GATED_D = 2.0 ** -20
# GELU: the argument z = 2v carries 5 roundings (g^2, two constants, the FMA,
# the product), an absolute error 5 u |z| of the exponent; act(g) flushes to
# zero for |z| > 87.3, so |z| counts up to there.
GELU_ARG_D = 6 * U
FLUSH = 1.2e-36


def e4m3_grid():
    v = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return np.array([x for x in v if x <= 448.0])


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = e4m3_grid()


def round_grid(v, grid):
    """Nearest signed grid value, ties to the entry of even index, held at the
    largest."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (hi % 2 == 0))
    return np.copysign(grid[np.where(up, hi, lo)], v)


def mx_exponent(amax, emax):
    """floor(log2 amax) - emax, clamped at -127; -127 for 0."""
    _, ex = np.frexp(amax)
    return np.where(amax > 0, np.maximum(ex - 1 - emax, -127), -127)


def decode_e4m3(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def unpack_e2m1(packed):
    """Packed codes [M, K/2] -> signed values [M, K]."""
    c = np.stack([packed & 15, packed >> 4], axis=-1).reshape(packed.shape[0], -1)
    return np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]


def mxfp4_quantize(x):
    """Values [M, K] (binary64) -> (packed codes, scale bytes [M, K/32])."""
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)
    e = mx_exponent(amax, 2)
    q = round_grid(np.where(bad[..., None], 0.0, b) * np.ldexp(1.0, -e)[..., None], E2M1)
    idx = np.searchsorted(E2M1, np.abs(q)).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 3)
    idx = np.where(bad[..., None], 7, idx).reshape(M, K).astype(np.uint8)
    return idx[:, 0::2] | (idx[:, 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def mxfp4_values(packed, scales):
    """Dequantized values [M, K] of packed codes and row-major scale bytes."""
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return unpack_e2m1(packed) * np.repeat(s, 32, axis=1)


def rmsnorm(h, w, eps):
    """y of the norm from the stored residual stream h, binary64."""
    h = h.double().cpu().numpy()
    return h * w.double().cpu().numpy() / np.sqrt((h * h).mean(-1, keepdims=True) + eps)


def gated(g, u, act):
    """(y, relative bound, absolute bound) of act(g) u, binary64."""
    g, u = g.double().cpu().numpy(), u.double().cpu().numpy()
    z = g if act == "silu" else 2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        a = np.where(z >= 0, g / (1.0 + np.exp(-np.abs(z))), g * np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
    d = GATED_D + (GELU_ARG_D * np.minimum(np.abs(z), 90.0) if act == "gelu_tanh" else 0.0)
    return a * u, np.broadcast_to(d, g.shape), FLUSH * np.abs(u) + 2.0 ** -148


def _between(got, v, slack, grid, what, typical=True):
    lo, hi = round_grid(v - slack, grid), round_grid(v + slack, grid)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} codes wrong, first at {np.argwhere(bad)[0]}: got "
                           f"{got[bad][0]}, value {v[bad][0]} (between {lo[bad][0]} and {hi[bad][0]})")
    if typical:
        # values anywhere between borders, which are at least 2^-4 of a value
        # apart: a slack of 2^-19 reaches one for 2 2^-19 / 2^-4 = 2^-14 of them,
        # so nearly every code must be the exact value's own.  (Not so for inputs
        # that sit on borders: with |g| < 2^-20, SiLU(g) = (g / 2)(1 + g / 2 ..) is
        # within the slack of g / 2, and a BF16 g / 2 is often half-way between
        # two E4M3 codes.)
        same = float(np.mean(got == round_grid(v, grid)))
        assert same > 0.999 or got.size < 5000, f"{what}: only {same:.5f} of the codes are the exact value's"


def check_mx(values, scale_bytes, y, d, extra=0.0, emax=8, grid=E4M3, what="", typical=True):
    """values: decoded codes [M, K]; scale_bytes row-major [M, K/32]; y binary64
    with relative bound d and absolute bound extra (arrays or numbers)."""
    M, K = y.shape
    slack = (np.abs(y) * d + extra) * np.ones_like(y)
    lo = np.maximum(np.abs(y) - slack, 0.0).reshape(M, -1, 32).max(-1)
    hi = (np.abs(y) + slack).reshape(M, -1, 32).max(-1)
    e = scale_bytes.astype(np.int64) - 127
    bad = ~((e >= mx_exponent(lo, emax)) & (e <= mx_exponent(hi, emax)))
    assert not bad.any(), f"{what}: {int(bad.sum())} block scales wrong, first at {np.argwhere(bad)[0]}"
    f = np.repeat(np.ldexp(1.0, -e), 32, axis=1)
    _between(values, y * f, slack * f, grid, what, typical)


def check_rowwise(values, s, y, d, extra=0.0, what=""):
    slack = (np.abs(y) * d + extra) * np.ones_like(y)
    lo, hi = np.maximum(np.abs(y) - slack, 0.0).max(-1) / 448.0, (np.abs(y) + slack).max(-1) / 448.0
    s = s.astype(np.float64)
    assert np.all((s >= lo * (1 - U) - 2.0 ** -149) & (s <= hi * (1 + U) + 2.0 ** -149)), f"{what}: row scales wrong"
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(s[:, None] > 0, y / s[:, None], 0.0)
        sl = np.where(s[:, None] > 0, slack / s[:, None] + U * np.abs(v), 0.0)
    _between(values, v, sl, E4M3, what)


def check_nvfp4(packed, scale_bytes, g, y, d, extra=0.0, what=""):
    """scale_bytes row-major [M, K/16], g the global scale."""
    M, K = y.shape
    slack = (np.abs(y) * d + extra) * np.ones_like(y)
    gs = np.float64(np.float32(g) / np.float32(6.0))
    lo = np.maximum(np.abs(y) - slack, 0.0).reshape(M, -1, 16).max(-1) * gs
    hi = (np.abs(y) + slack).reshape(M, -1, 16).max(-1) * gs
    s = decode_e4m3(scale_bytes)
    assert np.all((s >= round_grid(lo * (1 - 2 * U), E4M3)) & (s <= round_grid(hi * (1 + 2 * U), E4M3))), \
        f"{what}: block scales wrong"
    with np.errstate(divide="ignore"):
        mul = np.where(s > 0, (np.float32(g) / s.astype(np.float32)).astype(np.float64), 0.0)
    mul = np.repeat(mul, 16, axis=1)
    _between(unpack_e2m1(packed), y * mul, (slack + 2 * U * np.abs(y)) * mul, E2M1, what)
