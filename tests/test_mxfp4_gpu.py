"""GPU parity of the MXFP4 layer: codes and scales bit-exact against the
64-bit form (a power-of-two scaling and one rounding on both sides), products
within the output tolerance of the exact result, the few-rows kernel and the
large one, and the calls a serving program makes (in-place buffers, other
streams, captured graphs)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fused_ref as ref
from helpers import assert_within_tol, bf16_bits, bf16_values, tc_bytes, unswizzle
from mxfp8_w8a8_quantized_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from mxfp8_w8a8_quantized_b200 import mxfp8
    return mxfp8


def _np(t):
    return t.detach().double().cpu().numpy()


def _check_quantized(codes, scales, v, M, K):
    rq, rs = ref.mxfp4_quantize(v)
    sc = scales.cpu().numpy()
    assert np.array_equal(unswizzle(sc, M, K), rs)
    assert np.array_equal(codes.cpu().numpy(), rq)
    pad = np.ones(tc_bytes(M, K), dtype=bool)
    from helpers import tc_index
    pad[tc_index(M, K)] = False
    assert not sc[:len(pad)][pad].any(), "padding scale bytes are not zero"


# (40000, 64): more rows than resident warps, whole rows per warp; (9000,
# 1056): rows in parts; odd numbers of blocks; one row, one block
@pytest.mark.parametrize("M,K", [(1, 32), (7, 5120), (129, 13824), (300, 1056), (64, 96), (9500, 1056), (40000, 64)])
def test_activation_quantizer_bit_exact(mx, M, K):
    x = synth.activations_device(M, K, M + K, 0, "cuda")
    codes = torch.full((M, K // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((mx.mxfp4_scale_bytes(M, K),), 0xAB, dtype=torch.uint8, device="cuda")
    mx.mxfp4_quantize(x, codes=codes, scales=scales)
    torch.cuda.synchronize()
    _check_quantized(codes, scales, _np(x), M, K)


def test_quantizer_edge_blocks_and_strides(mx):
    M, K = 12, 96
    big = synth.activations_device(M, 3 * K + 8, 3, 0, "cuda")
    x = big[:, K: 2 * K]
    x[1] = 0.0
    x[2, :32] = -0.0
    x[3, 32:64] = 1e-40                          # a BF16 subnormal
    x[4, 5] = 3.3e38                             # near the largest
    x[5, 7] = float("inf")
    x[6, 70] = float("nan")
    x[7, 0] = float("-inf")
    x[8, :32] = 2.0 ** -126
    x[9, :32] = 5.0                              # a tie, and amax a power of two below
    x[10, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4)
    codes, scales = mx.mxfp4_quantize(x)
    c2, s2 = mx.mxfp4_quantize(x.contiguous())
    torch.cuda.synchronize()
    _check_quantized(codes, scales, _np(x), M, K)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


@pytest.mark.parametrize("N,K", [(512, 512), (333, 13824), (8, 32), (136, 1056)])
def test_weight_quantizer_bit_exact(mx, N, K):
    w = synth.weights_device(N, K, N + K, 0, "cuda")
    w[0, 0], w[N - 1, K - 1] = 1e-42, -3e38      # FP32 is not rounded to BF16 first
    codes, scales = mx.mxfp4_quantize_weight(w)
    torch.cuda.synchronize()
    _check_quantized(codes, scales, _np(w), N, K)


def test_no_rows(mx):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    codes, _ = mx.mxfp4_quantize(x)
    w = synth.weights_device(16, 64, 0, 0, "cuda")
    wq, ws = mx.mxfp4_quantize_weight(w)
    assert codes.shape == (0, 32) and mx.mxfp4_linear(x, wq, ws).shape == (0, 16)


# ------------------------------------------------------------------ GEMM
# Y within |Y - Yref| <= 2^-7 |Yref| + 1e-3 rms(Yref) of the exact result: one
# BF16 rounding (2^-8) and the FP32 accumulation.
def _layer(mx, M, K, N, seed, bias=True):
    x = synth.activations_device(M, K, seed, 0, "cuda")
    w = synth.weights_device(N, K, seed, 0, "cuda")
    b = synth.bias_device(N, seed, 0, "cuda") if bias else None
    return x, w, b, *mx.mxfp4_quantize_weight(w)


def _dequantized(t):
    """MXFP4 values of a tensor, on the GPU in FP64 (its 64-bit form)."""
    q, s = ref.mxfp4_quantize(_np(t))
    return torch.from_numpy(ref.mxfp4_values(q, s)).cuda()


def _reference(x, w, b):
    y = _dequantized(x) @ _dequantized(w).t()
    return (y if b is None else y + b.double()).cpu().numpy()


FEW = [(1, 32, 8), (1, 5120, 1384), (2, 256, 128), (16, 544, 264), (17, 544, 264), (31, 13824, 520), (33, 2080, 136),
       (64, 1024, 5120), (65, 4128, 136), (127, 96, 1000), (128, 2080, 1000), (5, 288, 40000)]
# more than one tile of rows in the few-rows kernel
FEW += [(129, 512, 512), (129, 32, 8), (300, 1056, 384), (1000, 1088, 1536), (517, 13824, 264), (260, 352, 520),
        (384, 5120, 5128)]
# more 128 x 128 tiles than SMs: the large kernel
MANY = [(2600, 512, 1024), (2000, 352, 1544), (1300, 13824, 2056), (4100, 96, 520), (20000, 32, 8), (129, 288, 19208)]


@pytest.mark.parametrize("M,K,N", FEW + MANY)
def test_gemm_within_tolerance(mx, M, K, N):
    x, w, b, wq, ws = _layer(mx, M, K, N, seed=M + N)
    xq, xs = mx.mxfp4_quantize(x)
    pad = torch.full((M + 1, N), -7.0, dtype=torch.bfloat16, device="cuda")
    y = mx.mxfp4_gemm(xq, xs, wq, ws, b, out=pad[:M])
    y2 = mx.mxfp4_linear(x, wq, ws, b)
    y3 = mx.mxfp4_gemm(xq, xs, wq, ws)
    torch.cuda.synchronize()
    assert mx.device_status() == 0
    assert torch.equal(y, y2), "mxfp4_linear differs from quantize + gemm"
    assert bool((pad[M] == -7.0).all()), "the row behind the output was written"
    assert_within_tol(bf16_values(bf16_bits(y)), _reference(x, w, b), f"mxfp4 {M}x{K}x{N}")
    assert_within_tol(bf16_values(bf16_bits(y3)), _reference(x, w, None), f"mxfp4 {M}x{K}x{N} without bias")


@pytest.mark.parametrize("M,K,N", [(1, 512, 136), (24, 288, 520), (90, 1056, 264), (130, 256, 136), (400, 800, 520),
                                   (3000, 288, 776), (2050, 544, 1288)])
def test_gemm_exact_on_grid_values(mx, M, K, N):
    """Values of the E2M1 grid with block scales of powers of two: every
    product and sum is exact in FP32 (multiples of 2^-6 below 2^18), so Y is the
    BF16 rounding of the exact result -- a misplaced scale or code shows."""
    gen = torch.Generator(device="cpu").manual_seed(M + K)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])

    def make(rows):
        v = grid[torch.randint(0, 8, (rows, K), generator=gen)]
        v = v * torch.where(torch.rand((rows, K), generator=gen) < 0.5, -1.0, 1.0)
        v[:, ::32] = 6.0                          # the block's scale is then exactly 1
        e = torch.randint(-2, 3, (rows, K // 32), generator=gen)
        return v * torch.ldexp(torch.ones(e.shape), e).repeat_interleave(32, dim=1)

    xv, wv = make(M), make(N)
    xq, xs = mx.mxfp4_quantize(xv.to(torch.bfloat16).cuda())
    wq, ws = mx.mxfp4_quantize_weight(wv.cuda())
    y = mx.mxfp4_gemm(xq, xs, wq, ws)
    torch.cuda.synchronize()
    exact = xv.double() @ wv.double().t()
    assert float(exact.abs().max()) < 2 ** 18
    assert torch.equal(y.cpu(), exact.to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("M,N", [(3, 264), (200, 264), (3000, 776)])
def test_gemm_nan_stays_in_its_row_and_column(mx, M, N):
    K = 544
    x, w, b, wq, ws = _layer(mx, M, K, N, 5)
    want = mx.mxfp4_linear(x, wq, ws, b)
    x2, w2 = x.clone(), w.clone()
    x2[1, 40] = float("nan")
    w2[77, 500] = float("inf")
    got = mx.mxfp4_linear(x2, *mx.mxfp4_quantize_weight(w2), b)
    torch.cuda.synchronize()
    hit = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    hit[1], hit[:, 77] = True, True
    assert torch.equal(torch.isnan(got), hit)
    assert torch.equal(got[~hit], want[~hit])


def test_gemm_repeats_bit_for_bit(mx):
    for M in (1, 40, 128, 300, 2600):
        x, w, b, wq, ws = _layer(mx, M, 4128, 1032, M)
        ys = [mx.mxfp4_linear(x, wq, ws, b) for _ in range(5)]
        torch.cuda.synchronize()
        assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_rows_do_not_depend_on_the_batch(mx):
    """A token's result is the same whatever tokens share its call, where the
    calls split K alike (eight weight tiles of nine K steps: eight parts)."""
    x, w, b, wq, ws = _layer(mx, 128, 2080, 1000, 9)
    whole = mx.mxfp4_linear(x, wq, ws, b)
    for M in (1, 16, 17, 64, 100):
        assert torch.equal(mx.mxfp4_linear(x[:M], wq, ws, b), whole[:M])


def test_two_streams_and_captured_graphs(mx):
    """Layers on two streams at once, each with a workspace of its own, and
    each captured into a graph that is replayed on new inputs."""
    for M in (4, 200, 2300):
        K, N = 2080, 1032
        runs = []
        for i in range(2):
            x, w, b, wq, ws = _layer(mx, M, K, N, 20 + i)
            wk = torch.empty(mx.mxfp4_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
            runs.append((x, wq, ws, b, wk, mx.mxfp4_linear(x, wq, ws, b), torch.cuda.Stream()))
        torch.cuda.synchronize()
        outs = [[], []]
        for _ in range(10):
            for i, (x, wq, ws, b, wk, _, st) in enumerate(runs):
                with torch.cuda.stream(st):
                    outs[i].append(mx.mxfp4_linear(x, wq, ws, b, workspace=wk))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(o, runs[i][5]) for o in outs[i])
        graphs = []
        for x, wq, ws, b, wk, _, _ in runs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                y = mx.mxfp4_linear(x, wq, ws, b, workspace=wk)
            graphs.append((g, y))
        for step in range(3):
            for i, (x, *_rest) in enumerate(runs):
                x.copy_(synth.activations_device(M, K, 50 + 2 * step + i, 0, "cuda"))
            torch.cuda.synchronize()
            for (g, _), r in zip(graphs, runs):
                with torch.cuda.stream(r[6]):
                    g.replay()
            torch.cuda.synchronize()
            for (_, y), (x, wq, ws, b, *_rest) in zip(graphs, runs):
                assert torch.equal(y, mx.mxfp4_linear(x, wq, ws, b))
        torch.cuda.synchronize()
    assert mx.device_status() == 0


def test_weights_written_just_before_the_layer(mx):
    """The layer reads weights that the work right ahead of it on the stream
    wrote: nothing it loads early may be stale."""
    M, K, N = 2, 4096, 2048
    x, w0, b, wq0, ws0 = _layer(mx, M, K, N, 31)
    _, w1, _, wq1, ws1 = _layer(mx, M, K, N, 32)
    want = [mx.mxfp4_linear(x, wq0, ws0, b), mx.mxfp4_linear(x, wq1, ws1, b)]
    wq, ws = wq0.clone(), ws0.clone()
    got = []
    for i in range(20):
        s, t = ((wq0, ws0), (wq1, ws1))[i & 1]
        wq.copy_(s)
        ws.copy_(t)
        got.append(mx.mxfp4_linear(x, wq, ws, b))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i & 1])


def test_gemm_full_size_sampled(mx):
    """M = 32760 at the Q projection's widths: sampled outputs."""
    M, K, N = synth.TOKENS_480P, synth.HIDDEN, synth.HIDDEN
    x, w, b, wq, ws = _layer(mx, M, K, N, 1)
    y = mx.mxfp4_linear(x, wq, ws, b)
    torch.cuda.synchronize()
    assert mx.device_status() == 0
    rng = np.random.default_rng(0)
    rows = np.unique(np.concatenate([[0, 127, 128, 255, 256, M - 129, M - 1], rng.choice(M, 200, replace=False)]))
    rows = torch.from_numpy(rows).cuda()
    assert_within_tol(bf16_values(bf16_bits(y[rows])), _reference(x[rows], w, b), "mxfp4 Q projection")


def test_binding_refuses_wrong_shapes(mx):
    x, w, b, wq, ws = _layer(mx, 4, 64, 16, 0)
    xq, xs = mx.mxfp4_quantize(x)
    for call in (lambda: mx.mxfp4_gemm(xq, xs[:100], wq, ws),
                 lambda: mx.mxfp4_gemm(xq, xs, wq, ws[:100]),
                 lambda: mx.mxfp4_gemm(xq[:, :16].contiguous(), xs, wq, ws),
                 lambda: mx.mxfp4_gemm(xq, xs, wq, ws, b[:8]),
                 lambda: mx.mxfp4_gemm(xq, xs, wq, ws, b.float()),
                 lambda: mx.mxfp4_gemm(xq, xs, wq, ws, out=torch.empty((4, 8), dtype=torch.bfloat16, device="cuda")),
                 lambda: mx.mxfp4_linear(x[:, :32].contiguous(), wq, ws),
                 lambda: mx.mxfp4_linear(x.float(), wq, ws),
                 lambda: mx.mxfp4_quantize(x, codes=torch.empty((4, 16), dtype=torch.uint8, device="cuda")),
                 lambda: mx.mxfp4_quantize(x.t()),
                 lambda: mx.mxfp4_quantize(x, scales=torch.empty(100, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mx.MXFP8Error):
        mx.mxfp4_linear(x, wq, ws, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mx.MXFP8Error):
        mx.mxfp4_quantize(torch.zeros((4, 48), dtype=torch.bfloat16, device="cuda"))


def test_wait_gives_up_and_the_layer_runs_on(mx):
    mx.selftest_wait_timeout(mx.SELFTEST_MXFP4_FEW_ROWS, 1_000_000)
    assert mx.device_status() == 5
    assert mx.device_status() == 0
    x, w, b, wq, ws = _layer(mx, 3, 256, 64, 2)
    assert_within_tol(bf16_values(bf16_bits(mx.mxfp4_linear(x, wq, ws, b))), _reference(x, w, b))


def test_large_gemm_single_cta_variant_in_subprocess():
    # the large GEMM's single-CTA variant is fixed per process
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, MXFP8_GEMM_PAIR="0")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        os.path.join(here, "test_mxfp4_gpu.py"), "-k", "within_tolerance or grid_values or nan_stays"],
                       env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
