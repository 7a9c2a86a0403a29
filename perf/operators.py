"""Cases of the operators around a quantized linear layer: the residual + RMS
norm that writes the layer's quantized input, the gated activation that does
so between a feed-forward pair, the MXFP4 linear layer itself, and the four
of them in a row as a gated feed-forward block.

A case is a dict with an "op":

  norm    h = BF16(x + residual); y = h weight / sqrt(mean(h^2) + eps), y
          quantized to 8 bits: MXFP8 (E4M3 codes, one E8M0 scale per 32
          elements, tensor-core layout) or per-channel FP8 (E4M3 codes, one
          FP32 scale per row)
  gated   y = act(gate) up, gate and up the two halves of a fused
          projection's output, quantized in the same ways
  linear  Y = BF16(x W^T + bias) with both operands in MXFP4 (E2M1 codes, one
          E8M0 scale per 32 elements); x is quantized within the call
  mlp     norm (MXFP4 output) -> gate/up product -> gated (MXFP4 output) ->
          down product
"""
import math

import torch

own = False

EPS = 1e-6
HIDDEN, FFN = 5120, 13824       # this repository's widths
DEVICE = "cuda"


def listed():
    return [
        # one token of a decoding step: latency, not bandwidth
        {"name": "norm_mxfp8_1x5120", "op": "norm", "fmt": "mxfp8", "M": 1, "K": HIDDEN, "residual": True},
        # a batch of prompts of odd total length
        {"name": "norm_fp8rw_4099x5120", "op": "norm", "fmt": "fp8rw", "M": 4099, "K": HIDDEN, "residual": True},
        # the first norm of a stack (nothing to add yet), a width that ends inside a scale atom
        {"name": "norm_mxfp8_777x4128", "op": "norm", "fmt": "mxfp8", "M": 777, "K": 4128, "residual": False},
        # all video tokens of an 832x1104 clip
        {"name": "norm_mxfp8_75348x5120", "op": "norm", "fmt": "mxfp8", "M": 75348, "K": HIDDEN, "residual": True},
        # a few sequences decoded together
        {"name": "gated_mxfp8_7x13824", "op": "gated", "fmt": "mxfp8", "act": "silu", "M": 7, "K": FFN},
        # a prompt, one scale per token: the row's maximum is needed before its first code
        {"name": "gated_fp8rw_2047x13824", "op": "gated", "fmt": "fp8rw", "act": "gelu_tanh", "M": 2047, "K": FFN},
        # all tokens of a 480p clip
        {"name": "gated_mxfp8_32760x13824", "op": "gated", "fmt": "mxfp8", "act": "silu", "M": 32760, "K": FFN},
        # a decoding step's up projection: one token against the whole weight
        {"name": "linear_mxfp4_1x5120x13824", "op": "linear", "M": 1, "K": HIDDEN, "N": FFN, "bias": False},
        # a decoding batch's down projection: long K, few rows
        {"name": "linear_mxfp4_33x13824x5120", "op": "linear", "M": 33, "K": FFN, "N": HIDDEN, "bias": True},
        # an odd prompt on a width that is not a multiple of the scale atom
        {"name": "linear_mxfp4_1021x4128x5128", "op": "linear", "M": 1021, "K": 4128, "N": 5128, "bias": True},
        # the 480p clip's feed-forward projection
        {"name": "linear_mxfp4_32760x5120x13824", "op": "linear", "M": 32760, "K": HIDDEN, "N": FFN, "bias": True},
        # the block as it is used while decoding a batch
        {"name": "mlp_mxfp4_16x5120x13824", "op": "mlp", "act": "silu", "M": 16, "K": HIDDEN, "N": FFN},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "gated", "linear", "linear", "mlp"))
    if op == "norm":
        K = 32 * _log_int(rng, 2, 512)
        return {"op": op, "fmt": rng.choice(("mxfp8", "fp8rw")), "M": _log_int(rng, 1, min(75348, 75348 * HIDDEN // K)),
                "K": K, "residual": rng.random() < 0.7}
    if op == "gated":
        K = 32 * _log_int(rng, 2, 512)
        return {"op": op, "fmt": rng.choice(("mxfp8", "fp8rw")), "act": rng.choice(("silu", "gelu_tanh")),
                "M": _log_int(rng, 1, min(75348, 32760 * FFN // K)), "K": K}
    if op == "linear":
        return {"op": op, "M": _log_int(rng, 1, 32760), "K": 32 * _log_int(rng, 2, 160), "N": 8 * _log_int(rng, 4, 1728),
                "bias": rng.random() < 0.5}
    return {"op": op, "act": rng.choice(("silu", "gelu_tanh")), "M": _log_int(rng, 1, 2048),
            "K": 32 * _log_int(rng, 8, 160), "N": 32 * _log_int(rng, 8, 432)}


# ------------------------------------------------------------------- inputs
def _gen(seed, tag):
    g = torch.Generator(device=DEVICE)
    g.manual_seed((int(seed) * 1_000_003 + tag * 10_007) & 0x7FFF_FFFF_FFFF)
    return g


def _activations(M, K, seed, tag):
    """BF16 N(0, 1) with 1 % of the channels twenty times as large (the
    outlier channels of a transformer's hidden state); one row in 61 is
    zero, as the padding of a batch is."""
    g = _gen(seed, tag)
    x = torch.randn(M, K, generator=g, dtype=torch.float32, device=DEVICE)
    x[:, torch.randperm(K, generator=g, device=DEVICE)[: max(1, K // 100)]] *= 20.0
    x[60::61] = 0.0
    return x.to(torch.bfloat16)


def _tc_offsets(rows, K):
    """Byte offset of every (row, 32-element block) scale in the tensor-core
    layout: 512-byte atoms of 128 rows x 4 blocks, and the array's bytes."""
    nb = K // 32
    groups = (nb + 3) // 4
    r = torch.arange(rows, device=DEVICE)[:, None]
    b = torch.arange(nb, device=DEVICE)[None, :]
    at = ((r // 128) * groups + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    return at, (rows + 127) // 128 * groups * 512


def _mxfp4_weight(N, K, seed, tag):
    """N(0, 1/sqrt(K)) weights in MXFP4 as a program keeps them: packed E2M1
    codes [N, K/2] (even element in the low nibble) and E8M0 scales in the
    tensor-core layout."""
    w = torch.randn(N, K, generator=_gen(seed, tag), dtype=torch.float32, device=DEVICE) * (1.0 / math.sqrt(K))
    blocks = w.view(N, K // 32, 32)
    e = _exponent(blocks.abs().amax(-1), 2)
    a = blocks.abs() * _pow2(-e)[..., None]
    idx = _e2m1_index(a) + 8 * torch.signbit(blocks).to(torch.uint8)
    idx = idx.view(N, K)
    codes = (idx[:, 0::2] | (idx[:, 1::2] << 4)).contiguous()
    at, size = _tc_offsets(N, K)
    scales = torch.zeros(size, dtype=torch.uint8, device=DEVICE)
    scales[at] = (e + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    s = dict(case)
    M, K = case["M"], case["K"]
    if case["op"] in ("norm", "mlp"):
        s["x"] = _activations(M, K, seed, 1)
        s["r"] = _activations(M, K, seed, 2) if case.get("residual", True) else None
        s["w"] = (1.0 + 0.1 * torch.randn(K, generator=_gen(seed, 3), device=DEVICE)).to(torch.bfloat16)
    if case["op"] == "gated":
        gu = _activations(M, 2 * K, seed, 4)    # a fused projection's output
        s["gate"], s["up"] = gu[:, :K], gu[:, K:]
    if case["op"] == "linear":
        N = case["N"]
        s["x"] = _activations(M, K, seed, 5)
        s["wq"], s["ws"] = _mxfp4_weight(N, K, seed, 6)
        s["b"] = None
        if case["bias"]:
            s["b"] = (0.01 * torch.randn(N, generator=_gen(seed, 7), device=DEVICE)).to(torch.float16)
    if case["op"] == "mlp":
        s["wq1"], s["ws1"] = _mxfp4_weight(2 * case["N"], K, seed, 8)
        s["wq2"], s["ws2"] = _mxfp4_weight(K, case["N"], seed, 9)
    return s


# --------------------------------------------------------------- plain forms
def _e2m1_index(a):
    """Nearest E2M1 magnitude (0, .5, 1, 1.5, 2, 3, 4, 6), ties to the even
    code, saturating: the number of borders below |a|."""
    n = (a > 0.25).to(torch.uint8)
    n += a >= 0.75
    n += a > 1.25
    n += a >= 1.75
    n += a > 2.5
    n += a >= 3.5
    n += a > 5.0
    return n


def _e2m1_value(idx):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEVICE)
    table = torch.cat([table, -table])
    return table[idx.long()]


def _exponent(amax, emax):
    """floor(log2 amax) - emax, held at the E8M0 minimum for an all-zero block."""
    e = torch.frexp(amax)[1] - 1 - emax
    return torch.where(amax > 0, e, -127).clamp_(min=-127)


def _pow2(e):
    """2^e exactly, for whole e in [-126, 127] (0 for -127, the exponent of an
    all-zero block)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _mxfp8(y):
    """(E4M3 codes, E8M0 scales in the tensor-core layout) of y [M, K]."""
    M, K = y.shape
    blocks = y.view(M, K // 32, 32)
    e = _exponent(blocks.abs().amax(-1), 8)
    codes = (blocks * _pow2(-e)[..., None]).clamp_(-448.0, 448.0).view(M, K).to(torch.float8_e4m3fn)
    at, size = _tc_offsets(M, K)
    scales = torch.zeros(size, dtype=torch.uint8, device=DEVICE)
    scales[at] = (e + 127).to(torch.uint8)
    return codes, scales.view(torch.float8_e8m0fnu)


def _fp8rw(y):
    """(E4M3 codes, FP32 scale of each row) of y [M, K]; an all-zero row has
    scale 0 and zero codes."""
    s = y.abs().amax(-1) / 448.0
    q = torch.where(s[:, None] > 0, y / s[:, None], y)
    return q.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _mxfp4_dequantized(y):
    """y rounded to MXFP4, as values."""
    M, K = y.shape
    blocks = y.view(M, K // 32, 32)
    e = _exponent(blocks.abs().amax(-1), 2)[..., None]
    a = blocks * _pow2(-e)
    v = _e2m1_value(_e2m1_index(a.abs()))
    return (torch.copysign(v, a) * _pow2(e)).view(M, K)


def _mxfp4_weight_values(wq, ws):
    N, K = wq.shape[0], wq.shape[1] * 2
    idx = torch.stack([wq & 15, wq >> 4], dim=-1).view(N, K)
    at, _ = _tc_offsets(N, K)
    e = ws[at].to(torch.int32) - 127
    return (_e2m1_value(idx).view(N, K // 32, 32) * _pow2(e)[..., None]).view(N, K)


def _plain_norm(x, r, w):
    """(residual stream BF16, normalized y FP32)."""
    h = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    return h, f * w.float() * rstd


def _plain_gated(gate, up, act):
    g, u = gate.float(), up.float()
    if act == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    t = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)
    return g / (1.0 + torch.exp(-2.0 * t)) * u


def _plain_product(xv, wq, ws, b):
    y = xv @ _mxfp4_weight_values(wq, ws).t()
    if b is not None:
        y += b.float()
    return y.to(torch.bfloat16)


def _run_plain(s):
    quant = {"mxfp8": _mxfp8, "fp8rw": _fp8rw}
    if s["op"] == "norm":
        h, y = _plain_norm(s["x"], s["r"], s["w"])
        codes, scales = quant[s["fmt"]](y)
        return {"h": h if s["r"] is not None else None, "codes": codes, "scales": scales}
    if s["op"] == "gated":
        codes, scales = quant[s["fmt"]](_plain_gated(s["gate"], s["up"], s["act"]))
        return {"codes": codes, "scales": scales}
    if s["op"] == "linear":
        return {"y": _plain_product(_mxfp4_dequantized(s["x"].float()), s["wq"], s["ws"], s["b"])}
    h, y = _plain_norm(s["x"], s["r"], s["w"])
    gu = _plain_product(_mxfp4_dequantized(y), s["wq1"], s["ws1"], None)
    N = s["N"]
    a = _plain_gated(gu[:, :N], gu[:, N:], s["act"])
    return {"h": h, "y": _plain_product(_mxfp4_dequantized(a), s["wq2"], s["ws2"], None)}


# ------------------------------------------------------ the framework's calls
def _run_own(s):
    from mxfp8_w8a8_quantized_b200 import mxfp8 as mx
    act = {"silu": mx.ACT_SILU, "gelu_tanh": mx.ACT_GELU_TANH}
    if s["op"] == "norm":
        f = mx.rmsnorm_quantize if s["fmt"] == "mxfp8" else mx.fp8rw_rmsnorm_quantize
        codes, scales, h = f(s["x"], s["w"], EPS, residual=s["r"])
        return _eight_bit(s["fmt"], codes, scales, {"h": h if s["r"] is not None else None})
    if s["op"] == "gated":
        f = mx.gated_quantize if s["fmt"] == "mxfp8" else mx.fp8rw_gated_quantize
        codes, scales = f(s["gate"], s["up"], act[s["act"]])
        return _eight_bit(s["fmt"], codes, scales, {})
    if s["op"] == "linear":
        return {"y": mx.mxfp4_linear(s["x"], s["wq"], s["ws"], s["b"])}
    N = s["N"]
    codes, scales, h = mx.mxfp4_rmsnorm_quantize(s["x"], s["w"], EPS, residual=s["r"])
    gu = mx.mxfp4_gemm(codes, scales, s["wq1"], s["ws1"])
    codes, scales = mx.mxfp4_gated_quantize(gu[:, :N], gu[:, N:], act[s["act"]])
    return {"h": h, "y": mx.mxfp4_gemm(codes, scales, s["wq2"], s["ws2"])}


def _eight_bit(fmt, codes, scales, out):
    """The 8-bit outputs as the values they stand for."""
    out["codes"] = codes.view(torch.float8_e4m3fn)
    out["scales"] = scales.view(torch.float8_e8m0fnu) if fmt == "mxfp8" else scales
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- accounting
def work(case):
    M, K = case["M"], case["K"]
    out = M * K * (1 + 1 / 32) if case.get("fmt") == "mxfp8" else M * K + 4 * M
    if case["op"] == "norm":
        streams = 3 if case["residual"] else 1      # x, residual and their sum; or x alone
        return {"bytes": 2 * M * K * streams + 2 * K + out, "flops": 6 * M * K}
    if case["op"] == "gated":
        return {"bytes": 4 * M * K + out, "flops": 8 * M * K}
    N = case["N"]
    if case["op"] == "linear":
        return {"bytes": 2 * M * K + N * K * (1 / 2 + 1 / 32) + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    return {"bytes": 8 * M * K + 2 * K + 3 * N * K * (1 / 2 + 1 / 32), "flops": 6 * M * N * K}


# ------------------------------------------------------- 64-bit definitions
def _round_to(v, grid):
    """Nearest entry of an increasing grid of non-negative values, ties to
    the entry of even index, values beyond the last held there."""
    hi = torch.searchsorted(grid, v.contiguous()).clamp_(1, grid.numel() - 1)
    lo = hi - 1
    below, above = v - grid[lo], grid[hi] - v
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[torch.where(up, hi, lo)]


def _grid(exponents, mantissa_bits, last):
    """0, the subnormals and the normal values of a small float format."""
    n = 2 ** mantissa_bits
    v = [m / n * 2.0 ** exponents[0] for m in range(n)]
    v += [(1 + m / n) * 2.0 ** e for e in exponents for m in range(n)]
    return torch.tensor([x for x in v if x <= last], dtype=torch.float64, device=DEVICE)


def _two_to(e):
    """2^e in binary64, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_mx(y, grid, emax):
    """(values on the grid, scale exponents) of y in blocks of 32."""
    b = y.reshape(y.shape[0], -1, 32)
    top = b.abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(_two_to(e) > top, e - 1, e)         # log2 rounded to a whole number
    e = torch.where(_two_to(e + 1) <= top, e + 1, e)
    e = torch.where(top > 0, (e - emax).clamp(min=-127), -127.0)
    q = b / _two_to(e)[..., None]
    return torch.copysign(_round_to(q.abs().reshape(-1), grid).view_as(q), q).view_as(y), e


def _exact_norm(s):
    x = s["x"].double()
    h = x if s["r"] is None else (x + s["r"].double()).to(torch.bfloat16).double()
    return h, h * s["w"].double() / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + EPS)


def _exact_gated(g, u, act):
    if act == "silu":
        return g * torch.sigmoid(g) * u
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u


def _exact_eight_bit(y, fmt):
    grid = _grid(range(-6, 9), 3, 448.0)
    if fmt == "fp8rw":
        sc = y.abs().amax(-1, keepdim=True) / 448.0
        q = torch.where(sc > 0, y / sc, y)
        return torch.copysign(_round_to(q.abs().reshape(-1), grid).view_as(q), q), sc[:, 0]
    codes, e = _exact_mx(y, grid, 8)
    at, size = _tc_offsets(*y.shape)
    scales = torch.full((size,), 2.0 ** -127, dtype=torch.float64, device=DEVICE)
    scales[at] = _two_to(e)
    return codes, scales


def _exact_mxfp4(y):
    v, e = _exact_mx(y, _grid(range(0, 3), 1, 6.0), 2)
    return (v.view(y.shape[0], -1, 32) * _two_to(e)[..., None]).view_as(y)


def _exact_weight(wq, ws):
    N = wq.shape[0]
    n = torch.stack([wq % 16, wq // 16], dim=-1).reshape(N, -1).long()
    m, ex, sign = n % 2, (n // 2) % 4, n // 8
    mag = torch.where(ex == 0, m * 0.5, (1.0 + 0.5 * m) * _two_to(ex - 1))
    at, _ = _tc_offsets(N, n.shape[1])
    sc = _two_to(ws[at].to(torch.int64) - 127)
    return ((1 - 2 * sign) * mag * sc.repeat_interleave(32, dim=1))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h, y = _exact_norm(s)
        codes, scales = _exact_eight_bit(y, case["fmt"])
        return {"h": h if s["r"] is not None else None, "codes": codes, "scales": scales}
    if case["op"] == "gated":
        codes, scales = _exact_eight_bit(_exact_gated(s["gate"].double(), s["up"].double(), case["act"]), case["fmt"])
        return {"codes": codes, "scales": scales}
    if case["op"] == "linear":
        y = _exact_mxfp4(s["x"].double()) @ _exact_weight(s["wq"], s["ws"]).t()
        return {"y": y if s["b"] is None else y + s["b"].double()}
    h, y = _exact_norm(s)
    gu = (_exact_mxfp4(y) @ _exact_weight(s["wq1"], s["ws1"]).t()).to(torch.bfloat16).double()
    a = _exact_gated(gu[:, : case["N"]], gu[:, case["N"]:], case["act"])
    return {"h": h, "y": _exact_mxfp4(a) @ _exact_weight(s["wq2"], s["ws2"]).t()}
