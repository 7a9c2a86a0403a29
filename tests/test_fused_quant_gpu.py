"""GPU parity of the RMS norm and the gated activation with quantized output,
in every format, against their 64-bit forms (fused_ref: a code is right when
it lies between those of y (1 - d) and y (1 + d), d the derived binary32 error
bound), and a gated feed-forward block of them with the MXFP4 products."""
import numpy as np
import pytest
import torch

import fused_ref as ref
from helpers import assert_within_tol, bf16_bits, bf16_values, tc_index, unswizzle
from mxfp8_w8a8_quantized_b200 import synth

pytestmark = pytest.mark.gpu
EPS = 1e-6
FORMATS = ("mxfp8", "mxfp8_rows", "fp8rw", "nvfp4", "mxfp4")


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def _g(v=37.5):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


def _norm(mx, fmt, x, w, **k):
    if fmt == "mxfp8":
        return mx.rmsnorm_quantize(x, w, EPS, **k)
    if fmt == "mxfp8_rows":
        return mx.rmsnorm_quantize(x, w, EPS, layout=mx.SF_ROWMAJOR, **k)
    if fmt == "nvfp4":
        return mx.nvfp4_rmsnorm_quantize(x, w, _g(), EPS, **k)
    return getattr(mx, f"{fmt}_rmsnorm_quantize")(x, w, EPS, **k)


def _gated(mx, fmt, g, u, act, **k):
    a = mx.ACT_SILU if act == "silu" else mx.ACT_GELU_TANH
    if fmt == "mxfp8":
        return mx.gated_quantize(g, u, a, **k)
    if fmt == "mxfp8_rows":
        return mx.gated_quantize(g, u, a, layout=mx.SF_ROWMAJOR, **k)
    if fmt == "nvfp4":
        return mx.nvfp4_gated_quantize(g, u, _g(), a, **k)
    return getattr(mx, f"{fmt}_gated_quantize")(g, u, a, **k)


def _check(fmt, codes, scales, y, d, extra=0.0, what=""):
    M, K = y.shape
    q, s = codes.cpu().numpy(), scales.cpu().numpy()
    if fmt == "fp8rw":
        return ref.check_rowwise(ref.decode_e4m3(q), s, y, d, extra, what)
    if fmt == "mxfp8_rows":
        return ref.check_mx(ref.decode_e4m3(q), s.reshape(M, K // 32), y, d, extra, what=what)
    block = 16 if fmt == "nvfp4" else 32
    pad = np.ones((M + 127) // 128 * ((K + 4 * block - 1) // (4 * block)) * 512, dtype=bool)
    pad[tc_index(M, K, block)] = False
    assert not s[:len(pad)][pad].any(), f"{what}: padding scale bytes are not zero"
    rows = unswizzle(s, M, K, block)
    if fmt == "mxfp8":
        ref.check_mx(ref.decode_e4m3(q), rows, y, d, extra, what=what)
    elif fmt == "mxfp4":
        ref.check_mx(ref.unpack_e2m1(q), rows, y, d, extra, emax=2, grid=ref.E2M1, what=what)
    else:
        ref.check_nvfp4(q, rows, 37.5, y, d, extra, what)


def _buffers(fmt, mx, M, K):
    """Output buffers filled with a pattern, so that nothing stays unwritten."""
    f = lambda *s: torch.full(s, 0xA5, dtype=torch.uint8, device="cuda")
    if fmt == "fp8rw":
        return dict(codes=f(M, K), scales=torch.full((M,), -3.0, device="cuda"))
    if fmt == "mxfp8_rows":
        return dict(codes=f(M, K), scales=f(M * K // 32))
    if fmt == "mxfp8":
        return dict(codes=f(M, K), scales=f(mx.scale_bytes(M, K)))
    return dict(codes=f(M, K // 2), scales=f((mx.nvfp4_scale_bytes if fmt == "nvfp4" else mx.mxfp4_scale_bytes)(M, K)))


def _inputs(M, K, seed, dtype=torch.bfloat16):
    x = synth.activations_device(M, K, seed, 0, "cuda")
    r = synth.activations_device(M, K, seed, 1, "cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(dtype)
    return x, r, w


# rows shorter and longer than each variant's reach, a row that ends inside a
# scale word or a warp, one block, many rows per CTA
NORM_SHAPES = [(1, 32), (1, 5120), (3, 96), (130, 2048), (65, 2080), (257, 5120), (100, 5152), (33, 8192), (9, 8224),
               (5, 16384), (20000, 64)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm_matches_the_formula(mx, fmt, M, K):
    x, r, w = _inputs(M, K, M + K)
    x[M // 2] = 0.0                                # a padding row
    r[M // 2] = 0.0
    codes, scales, h = _norm(mx, fmt, x, w, residual=r, **_buffers(fmt, mx, M, K))
    torch.cuda.synchronize()
    assert torch.equal(h, (x.double() + r.double()).to(torch.bfloat16))
    _check(fmt, codes, scales, ref.rmsnorm(h, w, EPS), ref.NORM_D, what=f"{fmt} {M}x{K}")
    codes, scales, h = _norm(mx, fmt, x, w, **_buffers(fmt, mx, M, K))
    torch.cuda.synchronize()
    assert h is x
    _check(fmt, codes, scales, ref.rmsnorm(x, w, EPS), ref.NORM_D, what=f"{fmt} {M}x{K} without residual")


@pytest.mark.parametrize("K", [8, 24, 5128, 13832])
def test_norm_rowwise_any_multiple_of_8(mx, K):
    x, r, w = _inputs(19, K, K)
    codes, scales, h = mx.fp8rw_rmsnorm_quantize(x, w, EPS, residual=r)
    torch.cuda.synchronize()
    _check("fp8rw", codes, scales, ref.rmsnorm(h, w, EPS), ref.NORM_D)


@pytest.mark.parametrize("K", [16, 48, 5136])
def test_norm_nvfp4_any_multiple_of_16(mx, K):
    x, r, w = _inputs(19, K, K)
    codes, scales, h = mx.nvfp4_rmsnorm_quantize(x, w, _g(), EPS, residual=r)
    torch.cuda.synchronize()
    _check("nvfp4", codes, scales, ref.rmsnorm(h, w, EPS), ref.NORM_D)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", ("mxfp8", "fp8rw"))
def test_norm_weight_types(mx, fmt, dtype):
    x, r, w = _inputs(37, 1056, 3, dtype)
    codes, scales, h = _norm(mx, fmt, x, w, residual=r)
    torch.cuda.synchronize()
    _check(fmt, codes, scales, ref.rmsnorm(h, w, EPS), ref.NORM_D)


@pytest.mark.parametrize("fmt", FORMATS)
def test_norm_strided_and_in_place(mx, fmt):
    M, K = 70, 544
    x, r, w = _inputs(M, K, 4)
    want = _norm(mx, fmt, x, w, residual=r)
    wide = torch.zeros((M, 3 * K + 16), dtype=torch.bfloat16, device="cuda")
    wide[:, K: 2 * K] = x
    rs = torch.zeros((M, 2 * K), dtype=torch.bfloat16, device="cuda")
    rs[:, :K] = r
    out = torch.full((M + 1, K + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    got = _norm(mx, fmt, wide[:, K: 2 * K], w, residual=rs[:, :K], residual_out=out[:M, :K])
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert bool((out[M] == 5.0).all()) and bool((out[:, K:] == 5.0).all())
    for which in ("x", "r"):                       # the stream updated in place
        a, b = x.clone(), r.clone()
        t = a if which == "x" else b
        got = _norm(mx, fmt, a, w, residual=b, residual_out=t)
        assert got[2] is t and all(torch.equal(p, q) for p, q in zip(want, got))


def test_norm_columns_of_one_buffer(mx):
    """x, residual and its sum may be column ranges of one buffer; ranges that
    share columns or rows are refused."""
    M, K = 40, 544
    x, r, w = _inputs(M, K, 5)
    want = mx.rmsnorm_quantize(x, w, EPS, residual=r)
    buf = torch.zeros((M + 1, 3 * K), dtype=torch.bfloat16, device="cuda")
    buf[:M, :K], buf[:M, 2 * K:] = x, r
    got = mx.rmsnorm_quantize(buf[:M, :K], w, EPS, residual=buf[:M, 2 * K:], residual_out=buf[:M, K: 2 * K])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for out in (buf[:M, 8: K + 8], buf[:M, 2 * K - 8: 3 * K - 8], buf[1:, :K], buf[:M, K + 8: 2 * K + 8]):
        with pytest.raises(ValueError):
            mx.rmsnorm_quantize(buf[:M, :K], w, EPS, residual=buf[:M, 2 * K:], residual_out=out)


def test_norm_weight_computed_by_the_kernel_ahead(mx):
    """An adaptive norm: the weight is what the product right ahead of it
    wrote, into the same buffer each time, with nothing waited for between."""
    M, K, E = 300, 1024, 256
    x, r, _ = _inputs(M, K, 11)
    wq, ws = mx.mxfp4_quantize_weight(synth.weights_device(K, E, 12, 0, "cuda"))
    emb = [synth.activations_device(1, E, 13 + i, 0, "cuda") for i in range(8)]
    want = []
    for e in emb:
        w = mx.mxfp4_linear(e, wq, ws)[0].clone()
        torch.cuda.synchronize()
        want.append(mx.rmsnorm_quantize(x, w, EPS, residual=r)[:2])
        torch.cuda.synchronize()
    buf = torch.empty((1, K), dtype=torch.bfloat16, device="cuda")
    for _ in range(10):
        got = []
        for e in emb:
            mx.mxfp4_linear(e, wq, ws, out=buf)
            got.append(mx.rmsnorm_quantize(x, buf[0], EPS, residual=r)[:2])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_large_offsets(mx):
    """Rows whose byte offsets pass 2^32 (a wide strided buffer)."""
    M, K, ld = 70000, 64, 32768
    wide = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    x = wide[:, :K]
    x.copy_(synth.activations_device(M, K, 6, 0, "cuda"))
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    a = mx.rmsnorm_quantize(x, w, EPS)
    b = mx.rmsnorm_quantize(x.contiguous(), w, EPS)
    c = mx.gated_quantize(x, wide[:, K: 2 * K].copy_(x), mx.ACT_SILU)
    d = mx.gated_quantize(x.contiguous(), x.contiguous(), mx.ACT_SILU)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])


def test_norm_values_that_are_not_finite(mx):
    M, K = 6, 128
    x, r, w = _inputs(M, K, 8)
    x[1, 40], x[2, 100] = float("nan"), float("inf")
    x[3] = 1e30                                    # the sum of squares overflows
    codes, scales, h = mx.rmsnorm_quantize(x, w, EPS)
    s = unswizzle(scales.cpu().numpy(), M, K)
    q = codes.cpu().numpy()
    assert np.all(s[1] == 255) and np.all(q[1] == 0x7F)
    assert s[2].tolist() == [0, 0, 0, 255] and np.all(q[2, 96:] == 0x7F) and not (q[2, :96] & 0x7F).any()
    assert not s[3].any() and not (q[3] & 0x7F).any()
    fine = [0, 4, 5]
    a, b, _ = mx.rmsnorm_quantize(x[fine], w, EPS)
    assert np.array_equal(q[fine], a.cpu().numpy())
    codes, scales, _ = mx.fp8rw_rmsnorm_quantize(x, w, EPS)
    assert bool(torch.isnan(scales[1])) and bool((codes[1] == 0x7F).all())
    assert float(scales[3]) == 0.0 and not bool((codes[3] & 0x7F).any())
    codes, scales, _ = mx.mxfp4_rmsnorm_quantize(x, w, EPS)
    s = unswizzle(scales.cpu().numpy(), M, K)
    assert np.all(s[1] == 255) and bool((codes[1] == 0x77).all()) and s[2].tolist() == [0, 0, 0, 255]


# ----------------------------------------------------------------- gated
GATED_SHAPES = [(1, 32), (7, 13824), (130, 2048), (3, 96), (65, 4128), (257, 2080), (33, 8224), (5, 16384), (20000, 64)]


@pytest.mark.parametrize("act", ("silu", "gelu_tanh"))
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", GATED_SHAPES)
def test_gated_matches_the_formula(mx, fmt, act, M, K):
    gu = synth.activations_device(M, 2 * K, M + K, 0, "cuda")
    gu[M // 2] = 0.0
    g, u = gu[:, :K], gu[:, K:]
    codes, scales = _gated(mx, fmt, g, u, act, **_buffers(fmt, mx, M, K))
    torch.cuda.synchronize()
    y, d, extra = ref.gated(g, u, act)
    _check(fmt, codes, scales, y, d, extra, f"{fmt} {act} {M}x{K}")
    c2, s2 = _gated(mx, fmt, g.contiguous(), u.contiguous(), act)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


@pytest.mark.parametrize("act", ("silu", "gelu_tanh"))
def test_gated_every_gate_value(mx, act):
    """Every finite BF16 gate up to 2^60 in magnitude, each in a block of its
    own magnitude, so that small results are seen too."""
    bits = torch.arange(0, 0x5D80, dtype=torch.int32)
    v = bits.to(torch.int16).view(torch.bfloat16)
    v = torch.cat([v, -v])
    g = v[:, None].expand(-1, 32).contiguous().cuda()
    u = torch.ones_like(g)
    codes, scales = mx.gated_quantize(g, u, mx.ACT_SILU if act == "silu" else mx.ACT_GELU_TANH)
    torch.cuda.synchronize()
    y, d, extra = ref.gated(g, u, act)
    rows = unswizzle(scales.cpu().numpy(), *y.shape)
    ref.check_mx(ref.decode_e4m3(codes.cpu().numpy()), rows, y, d, extra, what=act, typical=False)


def test_gated_values_that_are_not_finite(mx):
    M, K = 4, 128
    gu = synth.activations_device(M, 2 * K, 9, 0, "cuda")
    g, u = gu[:, :K].contiguous(), gu[:, K:].contiguous()
    want = mx.gated_quantize(g, u)
    g[0, 0], g[1, 40], u[2, 70], u[2, 100] = float("nan"), float("-inf"), float("inf"), float("nan")
    g[2, 70] = 1.0
    codes, scales = mx.gated_quantize(g, u)
    s, q = unswizzle(scales.cpu().numpy(), M, K), codes.cpu().numpy()
    hit = np.zeros((M, 4), dtype=bool)
    hit[0, 0] = hit[1, 1] = hit[2, 2] = hit[2, 3] = True
    assert np.array_equal(s == 255, hit)
    e = np.repeat(hit, 32, axis=1)
    assert np.all(q[e] == 0x7F) and np.array_equal(q[~e], want[0].cpu().numpy()[~e])


def test_no_rows(mx):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for fmt in FORMATS:
        assert _norm(mx, fmt, x, w, residual=x)[0].shape[0] == 0
        assert _gated(mx, fmt, x, x, "silu")[0].shape[0] == 0


def test_binding_refuses_wrong_shapes(mx):
    x, r, w = _inputs(4, 64, 0)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: mx.rmsnorm_quantize(x, w[:32]),
                 lambda: mx.rmsnorm_quantize(x, w.double()),
                 lambda: mx.rmsnorm_quantize(x.float(), w),
                 lambda: mx.rmsnorm_quantize(x, w, residual=r[:3]),
                 lambda: mx.rmsnorm_quantize(x, w, residual=r.float()),
                 lambda: mx.rmsnorm_quantize(x, w, residual_out=r),
                 lambda: mx.rmsnorm_quantize(x, w, residual=r, residual_out=bf(4, 32)),
                 lambda: mx.rmsnorm_quantize(x, w, codes=bf(4, 64)),
                 lambda: mx.rmsnorm_quantize(x, w, scales=torch.zeros(8, dtype=torch.uint8, device="cuda")),
                 lambda: mx.rmsnorm_quantize(x.t(), w[:4].contiguous()),
                 lambda: mx.fp8rw_rmsnorm_quantize(x, w, scales=torch.zeros(3, device="cuda")),
                 lambda: mx.nvfp4_rmsnorm_quantize(x, w, 1.0),
                 lambda: mx.gated_quantize(x, r[:, :32]),
                 lambda: mx.gated_quantize(x, r.half()),
                 lambda: mx.nvfp4_gated_quantize(x, r, torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    wide = bf(8, 64)                               # an output that overlaps its input row by row
    with pytest.raises(ValueError):
        mx.rmsnorm_quantize(wide[:4], w, residual=r, residual_out=wide[1:5])
    with pytest.raises(mx.MXFP8Error):
        mx.rmsnorm_quantize(x, w, eps=0.0)
    with pytest.raises(mx.MXFP8Error):
        mx.gated_quantize(x, r, act=mx.ACT_NONE)
    with pytest.raises(mx.MXFP8Error):
        mx.rmsnorm_quantize(x, w, layout=7)


# ----------------------------------------------- the operators together
def _block(mx, x, r, w, gate_up, down, act, out=None):
    """A gated feed-forward block in MXFP4: norm -> gate/up -> gated -> down."""
    N = gate_up[0].shape[0] // 2
    q, s, h = mx.mxfp4_rmsnorm_quantize(x, w, EPS, residual=r)
    gu = mx.mxfp4_gemm(q, s, *gate_up)
    a, t = mx.mxfp4_gated_quantize(gu[:, :N], gu[:, N:], act)
    return mx.mxfp4_gemm(a, t, *down, out=out), h, (q, s, gu, a, t)


@pytest.mark.parametrize("M", [1, 33, 300])
def test_feed_forward_block(mx, M):
    """Each step against its 64-bit form on the step's own input, and the
    block captured into a graph and replayed on new tokens."""
    K, N = 544, 1056
    x, r, w = _inputs(M, K, 40 + M)
    w1, w2 = synth.weights_device(2 * N, K, 41, 0, "cuda"), synth.weights_device(K, N, 42, 0, "cuda")
    gate_up, down = mx.mxfp4_quantize_weight(w1), mx.mxfp4_quantize_weight(w2)
    y, h, (q, s, gu, a, t) = _block(mx, x, r, w, gate_up, down, mx.ACT_SILU)
    torch.cuda.synchronize()
    assert mx.device_status() == 0
    _check("mxfp4", q, s, ref.rmsnorm(h, w, EPS), ref.NORM_D)
    val = lambda c, b, rows, cols: ref.mxfp4_values(c.cpu().numpy(), unswizzle(b.cpu().numpy(), rows, cols))
    exact = val(q, s, M, K) @ val(*gate_up, 2 * N, K).T
    assert_within_tol(bf16_values(bf16_bits(gu)), exact, "gate/up product")
    _check("mxfp4", a, t, *ref.gated(gu[:, :N], gu[:, N:], "silu"))
    exact = val(a, t, M, N) @ val(*down, K, N).T
    assert_within_tol(bf16_values(bf16_bits(y)), exact, "down product")

    out = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y2, h2, _ = _block(mx, x, r, w, gate_up, down, mx.ACT_SILU, out=out)
    for seed in (90, 91):
        x.copy_(synth.activations_device(M, K, seed, 0, "cuda"))
        r.copy_(synth.activations_device(M, K, seed, 1, "cuda"))
        graph.replay()
        y1, h1, _ = _block(mx, x, r, w, gate_up, down, mx.ACT_SILU)
        torch.cuda.synchronize()
        assert torch.equal(y1, y2) and torch.equal(h1, h2)


@pytest.mark.parametrize("M", [3, 129, 700])
def test_layers_over_the_same_buffers(mx, M):
    """Rows and gate/up halves that the kernel right ahead rewrites in place,
    layer after layer: a kernel that starts early asks for its first row before
    that, and must still see the new one.  Against the same steps, each waited for."""
    K, N = 544, 1056
    x, r, w = _inputs(M, K, 50)
    layers = [(mx.mxfp4_quantize_weight(synth.weights_device(2 * N, K, 51, i, "cuda")),
               mx.mxfp4_quantize_weight(synth.weights_device(K, N, 52, i, "cuda"))) for i in range(6)]

    def run(wait):
        y, h = x.clone(), r.clone()
        gu = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")
        pause = torch.cuda.synchronize if wait else (lambda: None)
        for up, down in layers:
            q, s, _ = mx.mxfp4_rmsnorm_quantize(y, w, EPS, residual=h, residual_out=h)
            pause()
            mx.mxfp4_gemm(q, s, *up, out=gu)
            pause()
            a, t = mx.mxfp4_gated_quantize(gu[:, :N], gu[:, N:], mx.ACT_SILU)
            pause()
            mx.mxfp4_gemm(a, t, *down, out=y)
            pause()
            mx.mxfp4_linear(y, *up, out=gu)     # the quantizer behind the product
            pause()
            y.add_(gu[:, :K])
            pause()
        return y, h

    want = run(True)
    assert torch.isfinite(want[0]).all()
    for _ in range(10):
        got = run(False)
        torch.cuda.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("M", [5, 2300])
def test_capture_with_fork_and_join(mx, M):
    """The operators in a captured graph behind copies, fills and work of other
    streams (each starts early only behind a kernel that lets it), replayed on
    new inputs; two such graphs share no memory and run at once."""
    K, N = 544, 1056
    x, r, w = _inputs(M, K, 70)
    gate_up = mx.mxfp4_quantize_weight(synth.weights_device(2 * N, K, 71, 0, "cuda"))
    down = mx.mxfp4_quantize_weight(synth.weights_device(K, N, 72, 0, "cuda"))
    src = torch.empty_like(x)

    def step(xs, rs, side):
        cur = torch.cuda.current_stream()
        xs.copy_(src)                                    # a copy ahead of the norm
        q, s, h = mx.mxfp4_rmsnorm_quantize(xs, w, EPS, residual=rs)
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            g = mx.mxfp4_gemm(q, s, gate_up[0][:N], gate_up[1])
        u = mx.mxfp4_linear(h, gate_up[0][:N].contiguous(), gate_up[1])
        cur.wait_stream(side)                            # two dependencies
        a, t = mx.mxfp4_gated_quantize(g, u, mx.ACT_GELU_TANH)
        out = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")    # a fill ahead of the product
        return mx.mxfp4_gemm(a, t, *down, out=out), h

    graphs = []
    for _ in range(2):
        xs, rs, side = torch.empty_like(x), r.clone(), torch.cuda.Stream()
        step(xs, rs, side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(xs, rs, side)
        graphs.append((graph, out, torch.cuda.Stream(), xs, rs))     # a graph's inputs have to live
    for seed in (3, 4, 5):
        src.copy_(synth.activations_device(M, K, seed, 0, "cuda"))
        torch.cuda.synchronize()
        for graph, _, st, *_ in graphs:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        y, h = step(torch.empty_like(x), r, torch.cuda.Stream())
        torch.cuda.synchronize()
        for _, (gy, gh), *_ in graphs:
            assert torch.equal(y, gy) and torch.equal(h, gh)


def test_first_calls_of_a_process_inside_a_capture():
    """No operator needs a call ahead of the capture: in a new process each is
    called for the first time while a graph is captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from mxfp8_w8a8_quantized_b200 import mxfp8 as mx
x = torch.randn(300, 512, device="cuda").bfloat16()
w = torch.ones(512, device="cuda")
big = torch.randn(4096, 512, device="cuda").bfloat16()
wt = torch.randn(1536, 512, device="cuda")
def run():
    wq, ws = mx.mxfp4_quantize_weight(wt)
    out = [mx.mxfp4_linear(big, wq, ws)]
    for M in (1, 20, 50, 300):
        q, s, h = mx.mxfp4_rmsnorm_quantize(x[:M], w, residual=x[:M])
        out += [h, mx.mxfp4_gemm(q, s, wq, ws), mx.mxfp4_linear(h, wq, ws)]
        out += list(mx.gated_quantize(h, x[:M])) + list(mx.fp8rw_gated_quantize(h, x[:M]))
        out += list(mx.fp8rw_rmsnorm_quantize(h, w))
    return out
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = run()
g.replay()
torch.cuda.synchronize()
b = run()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(a, b)) and mx.device_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]


def test_two_host_threads(mx):
    """Calls of several host threads, each on a stream of its own."""
    import threading
    K = 1056
    jobs = []
    for i in range(4):
        x, r, w = _inputs(33 + i, K, 80 + i)
        jobs.append((x, r, w, mx.rmsnorm_quantize(x, w, EPS, residual=r)))
    wq, ws = mx.mxfp4_quantize_weight(synth.weights_device(264, K, 81, 0, "cuda"))
    want = [mx.mxfp4_linear(j[0], wq, ws) for j in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        x, r, w, ref_out = jobs[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = mx.rmsnorm_quantize(x, w, EPS, residual=r)
                y = mx.mxfp4_linear(x, wq, ws)
                torch.cuda.current_stream().synchronize()
                if not (all(torch.equal(a, b) for a, b in zip(got, ref_out)) and torch.equal(y, want[i])):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_mxfp8_block_with_the_existing_gemm(mx):
    """The norm's and the gate's MXFP8 output is what the MXFP8 GEMM takes:
    the layer after them equals the GEMM on the reference's quantized input."""
    M, K, N = 200, 512, 384
    x, r, w = _inputs(M, K, 60)
    wq, ws = mx.quantize_weight(synth.weights_device(N, K, 61, 0, "cuda"))
    codes, scales, h = mx.rmsnorm_quantize(x, w, EPS, residual=r)
    y = mx.gemm_prequant(codes, scales, wq, ws)
    torch.cuda.synchronize()
    v = ref.decode_e4m3(codes.cpu().numpy()) * np.repeat(
        np.ldexp(1.0, unswizzle(scales.cpu().numpy(), M, K).astype(int) - 127), 32, axis=1)
    u = ref.decode_e4m3(wq.cpu().numpy()) * np.repeat(
        np.ldexp(1.0, unswizzle(ws.cpu().numpy(), N, K).astype(int) - 127), 32, axis=1)
    assert_within_tol(bf16_values(bf16_bits(y)), v @ u.T, "norm -> MXFP8 GEMM")
