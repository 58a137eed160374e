"""hstu_quant_groups_w4 and hstu_linear_w4_fwd against their definitions."""

import numpy as np
import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
from jagged_pointwise_attention_b200 import _native
from serving_util import U32, UBF, quant_w4_oracle, w4_values

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def ok():
    assert hstu.hstu_device_status() == _native.HSTU_OK


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 128), (7, 256), (130, 640), (2048, 512)])
def test_quant(G, N, K):
    rng = np.random.default_rng(N + K + G)
    W = torch.from_numpy(rng.standard_normal((N, K)) * rng.lognormal(0, 3, (N, 1))).to(BF)
    W[0, :G] = 0
    wide = torch.zeros(N, K + 6, dtype=BF)
    wide[:, 3:3 + K] = W
    codes, scales = hstu.hstu_quant_groups_w4(wide.cuda()[:, 3:3 + K], G)
    ok()
    wc, ws = quant_w4_oracle(W.double().numpy(), G)
    assert torch.equal(scales.cpu(), ws)
    assert np.array_equal(codes.cpu().numpy(), wc)


def test_quant_odd_values():
    """Zeros, the smallest and largest values, and groups that are not finite."""
    W = torch.zeros(6, 128, dtype=BF)
    W[1, 5] = 1e-40                              # its scale rounds to a subnormal or to zero
    W[2] = torch.finfo(BF).max
    W[3, 7], W[4, 9] = float("inf"), float("nan")
    W[5] = torch.linspace(-1, 1, 128).to(BF)
    codes, scales = hstu.hstu_quant_groups_w4(W.cuda(), 64)
    ok()
    c, s = codes.cpu().numpy(), scales.cpu()
    fine = [0, 1, 2, 5]
    wc, ws = quant_w4_oracle(W.double().numpy()[fine], 64)
    assert np.array_equal(c[fine], wc) and torch.equal(s[fine], ws)
    assert torch.isnan(s[3, 0]) and torch.isnan(s[4, 0]) and s[3, 1] == 1 and s[4, 1] == 1
    x = torch.ones(1, 128, dtype=BF).cuda()
    y = hstu.hstu_linear_w4_fwd(x, codes, scales).float().cpu()[0]
    assert torch.isnan(y[3]) and torch.isnan(y[4]) and torch.isfinite(y[[0, 1, 5]]).all()


def problem(M, K, N, G, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(BF)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = torch.from_numpy(rng.lognormal(-3, 1, (N, K // G))).to(BF)
    bias = torch.from_numpy(rng.standard_normal(N)).float()
    r = torch.from_numpy(rng.standard_normal((M, N))).to(BF)
    return x, codes, scales, bias, r


def check(y, x, codes, scales, G, bias, r, epilogue):
    """Products of a bf16 x and a 4-bit code are exact in fp32; the sum of K of
    them, the group scales and the bias are rounded in fp32 (at most two half
    steps a term), silu adds 8 half steps and the result is rounded to bf16."""
    W = w4_values(codes, scales, G)
    X = x.double().numpy()
    pre = X @ W.T
    err = (2 * X.shape[1] + 8) * U32 * (np.abs(X) @ np.abs(W).T + (0 if bias is None else np.abs(bias.double().numpy())))
    if bias is not None:
        pre = pre + bias.double().numpy()
    if epilogue == "silu":
        want = pre / (1 + np.exp(-pre))
        err = 1.1 * err + 8 * U32 * np.abs(want)
    elif epilogue == "residual":
        want = pre + r.double().numpy()
        err = err + 2 * U32 * np.abs(want)
    else:
        want = pre
    tol = err + UBF * (np.abs(want) + err) + 1e-30
    got = y.double().cpu().numpy()
    bad = np.abs(got - want) / tol
    assert bad.max() <= 1, bad.max()


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 130])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_linear_rows(M, G):
    K, N = 512, 200
    x, c, s, b, r = problem(M, K, N, G, M + G)
    ep = ("none", "silu", "residual")[(M + G // 32) % 3]
    y = hstu.hstu_linear_w4_fwd(x.cuda(), torch.from_numpy(c).cuda(), s.cuda(), b.cuda(), ep,
                                r.cuda() if ep == "residual" else None)
    ok()
    check(y, x, c, s, G, b, r, ep)


@pytest.mark.parametrize("K,N,M,G", [(128, 1, 1, 128), (128, 15, 3, 32), (256, 16, 1, 64),
                                     (384, 17, 5, 128), (640, 129, 8, 64), (2048, 31, 16, 128),
                                     (512, 2048, 1, 128), (8192, 500, 2, 128), (1152, 100, 64, 32),
                                     (16384, 40, 1, 128), (128, 5000, 40, 64)])
@pytest.mark.parametrize("epilogue", ["none", "silu", "residual"])
def test_linear_shapes(K, N, M, G, epilogue):
    x, c, s, b, r = problem(M, K, N, G, K + N)
    bias = None if N % 2 else b
    y = hstu.hstu_linear_w4_fwd(x.cuda(), torch.from_numpy(c).cuda(), s.cuda(),
                                None if bias is None else bias.cuda(), epilogue,
                                r.cuda() if epilogue == "residual" else None)
    ok()
    check(y, x, c, s, G, bias, r, epilogue)


def test_linear_strided_and_in_place_residual():
    M, K, N, G = 5, 256, 77, 64
    x, c, s, b, r = problem(M, K, N, G, 1)
    xw = torch.full((M, K + 24), float("nan"), dtype=BF).cuda()
    xw[:, 8:8 + K] = x.cuda()
    cw = torch.full((N, K // 2 + 32), 255, dtype=torch.uint8).cuda()
    cw[:, 16:16 + K // 2] = torch.from_numpy(c).cuda()
    sw = torch.full((N, K // G + 3), float("nan"), dtype=BF).cuda()
    sw[:, 1:1 + K // G] = s.cuda()
    yw = torch.full((M, N + 5), 3.0, dtype=BF).cuda()
    yw[:, 2:2 + N] = r.cuda()
    y = yw[:, 2:2 + N]
    hstu.hstu_linear_w4_fwd(xw[:, 8:8 + K], cw[:, 16:16 + K // 2], sw[:, 1:1 + K // G], b.cuda(),
                            "residual", y, out=y)
    ok()
    check(y, x, c, s, G, b, r, "residual")
    assert bool((yw[:, :2] == 3).all()) and bool((yw[:, 2 + N:] == 3).all())


def test_linear_no_rows_same_bits_and_graph():
    x, c, s, b, r = problem(8, 1024, 300, 128, 2)
    d = [x.cuda(), torch.from_numpy(c).cuda(), s.cuda(), b.cuda()]
    assert hstu.hstu_linear_w4_fwd(d[0][:0], *d[1:]).shape == (0, 300)
    want = hstu.hstu_linear_w4_fwd(*d)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hstu.hstu_linear_w4_fwd(*d, out=out)
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hstu.hstu_linear_w4_fwd(*d, stream=side)
    torch.cuda.synchronize()
    ok()
    assert torch.equal(out, want) and torch.equal(got, want)
    check(want, x, c, s, 128, b, r, "none")


def test_quantized_projection_close_to_the_weights():
    """The two together: a projection's error is the quantization's, at most half
    a scale a weight."""
    rng = np.random.default_rng(5)
    W = torch.from_numpy(rng.standard_normal((96, 512))).to(BF)
    x = torch.from_numpy(rng.standard_normal((4, 512))).to(BF)
    codes, scales = hstu.hstu_quant_groups_w4(W.cuda(), 64)
    y = hstu.hstu_linear_w4_fwd(x.cuda(), codes, scales)
    ok()
    X = np.abs(x.double().numpy())
    half = np.repeat(scales.double().cpu().numpy(), 64, axis=1) * (0.5 + 2.0 ** -8 * 8)
    want = x.double().numpy() @ W.double().numpy().T
    tol = X @ half.T
    tol = tol + UBF * (np.abs(want) + tol) + 1e-3
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [(33, 1024, 3190), (64, 1152, 3190), (65, 1024, 1600), (130, 2176, 1070),
                                   (40, 1024, 9490), (34, 256, 9490), (25, 256, 9490), (23, 1408, 300),
                                   (47, 896, 3190)])
def test_linear_many_rows(M, K, N, G):
    """More rows of x than a block of 32 takes: blocks of 64, and several blocks."""
    x, c, s, b, r = problem(M, K, N, G, M + K)
    ep = ("none", "silu", "residual")[(M + G // 32) % 3]
    y = hstu.hstu_linear_w4_fwd(x.cuda(), torch.from_numpy(c).cuda(), s.cuda(), b.cuda(), ep,
                                r.cuda() if ep == "residual" else None)
    ok()
    check(y, x, c, s, G, b, r, ep)
