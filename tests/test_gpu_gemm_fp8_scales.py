"""The 8-bit product where the product of two scales is no ordinary fp32 number.

Tolerance. That of test_gpu_gemm_fp8.py (each of a block's 128 additions off by 2^-23, two roundings for the scales, the blocks
added in fp32), and for each block 2^-125: a subnormal product of scales is off by 2^-150 at most, half of the
least subnormal, and a block's sums are below 128 * 448^2 < 2^25.
"""
import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from oracle import layer_ops as O

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
# Both kernels: 16, 32 and 64 rows of A to a tile, whole and shared reductions, tiles of 128 and of 256 columns.
SHAPES = [(3, 200, 400), (40, 333, 1744), (64, 1024, 2048), (333, 1000, 1744), (1, 4096, 4096), (512, 96, 128), (300, 520, 640),
          (600, 4100, 272), (1100, 9800, 384), (2000, 1500, 5200)]


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def product(dev, A, sA, W, sW):
    (M, K), N = A.shape, W.shape[0]
    d, Y = B.fo_gemm_fp8_desc(N, K, out_dtype="f32"), torch.full((M, N), 7.0, device=dev)
    ws = torch.empty(B.fo_gemm_fp8_workspace(d, M), dtype=torch.uint8, device=dev)
    B.fo_ops_workspace_init(ws)
    B.fo_gemm_fp8(d, M, [A.to(dev)], [sA.to(dev)], [W.to(dev)], [sW.to(dev)], [Y], ws)
    assert B.fo_ops_status_query(ws)[0] == 0
    return Y.cpu().double().numpy()


def operands(M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    draw = lambda *s: (8 + 440 * torch.rand(*s, generator=g)) * torch.where(torch.rand(*s, generator=g) < 0.5, -1.0, 1.0)  # noqa: E731
    A, W = draw(M, K).to(E4M3), draw(N, K).to(E4M3)
    kb = -(-K // 128)
    return A, torch.rand(M, kb, generator=g) + 0.5, W, torch.rand(-(-N // 128), kb, generator=g) + 0.5


def check(got, A, sA, W, sW):
    a, sa, w, sw = (t.double().numpy() for t in (A, sA, W, sW))
    want, size = O.gemm_fp8(a, sa, w, sw), O.gemm_fp8(np.abs(a), sa, np.abs(w), sw)
    n = sa.shape[1]
    assert np.all(np.abs(got - want) <= (128 * 2.0 ** -23 + (n + 4) * 2.0 ** -24) * size + n * 2.0 ** -125)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_whose_product_is_subnormal(dev, M, N, K):
    A, sA, W, sW = operands(M, N, K)
    for a, w in ((2e-38, 1e-4), (1e-4, 2e-38), (1e-20, 1e-21), (2.0 ** -126, 2.0 ** -30)):
        check(product(dev, A, sA * a, W, sW * w), A, sA * a, W, sW * w)
    # In every third row, in every second block: the other parts are as precise as ever.
    sA[::3] *= 1e-38
    sA[1::3, ::2] *= 1e-30
    check(product(dev, A, sA, W, sW * 1e-4), A, sA, W, sW * 1e-4)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_rows_of_zeros_under_the_least_scale(dev, M, N, K):
    # As the quantiser and the norm give them: values 0, scale 2^-126, beside ordinary rows.
    A, sA, W, sW = operands(M, N, K)
    A[::2], sA[::2] = 0.0, 2.0 ** -126
    got = product(dev, A, sA, W, sW * 1e-3)
    assert np.all(got[::2] == 0)
    check(got, A, sA, W, sW * 1e-3)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_whose_product_is_beyond_fp32_stay_in_their_row(dev, M, N, K):
    A, sA, W, sW = operands(M, N, K)
    sA[0, 0], sW[:, 0] = 1e30, sW[:, 0] * 1e20
    sA[1:, 0] *= 1e-20
    got = product(dev, A, sA, W, sW)
    assert not np.any(np.isfinite(got[0]))
    check(got[1:], A[1:], sA[1:], W, sW)
