"""The block-scaled product of 8-bit matrices against the fp64 oracle.

Tolerance. Products of two e4m3 values are exact in fp32. Within a block of 128 the tensor core adds them in an order and with a
rounding of its own: each addition counts as off by a whole step, 2^-23. Blocks are scaled (two roundings) and added
in fp32 (u = 2^-24 each). So a value is off by (128 * 2^-23 + (blocks + 3) * 2^-24) times the sum of the products'
magnitudes, and half a step of its type when it is stored. Whole-number inputs with scales that are powers of two are exact.
"""
import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from oracle import layer_ops as O

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


def operands(g, M, N, K, whole):
    kb = -(-K // 128)
    if whole:
        A, W = torch.randint(-4, 5, (M, K), generator=g).float(), torch.randint(-4, 5, (N, K), generator=g).float()
        sA = torch.exp2(torch.randint(-2, 3, (M, kb), generator=g).float())
        sW = torch.exp2(torch.randint(-2, 3, (-(-N // 128), kb), generator=g).float())
    else:
        A, W = 100 * torch.randn(M, K, generator=g), 100 * torch.randn(N, K, generator=g)
        sA, sW = torch.rand(M, kb, generator=g) + 0.01, 0.02 * torch.rand(-(-N // 128), kb, generator=g) + 1e-4
    return A.clamp(-448, 448).to(E4M3), sA, W.clamp(-448, 448).to(E4M3), sW


def product(dev, M, N, K, out, R=1, whole=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    ops = [operands(g, M, N, K, whole) for _ in range(R)]
    A, sA, W, sW = ([o[i].to(dev) for o in ops] for i in range(4))
    Y = [torch.full((M, N), float("nan"), dtype=TYPES[out], device=dev) for _ in range(R)]
    d = B.fo_gemm_fp8_desc(N, K, R=R, out_dtype=out)
    ws = torch.empty(B.fo_gemm_fp8_workspace(d, M), dtype=torch.uint8, device=dev)
    B.fo_ops_workspace_init(ws)
    B.fo_gemm_fp8(d, M, A, sA, W, sW, Y, ws)
    assert B.fo_ops_status_query(ws)[0] == 0
    for r in range(R):
        a, sa, w, sw = (f64(t) for t in ops[r])
        want = O.gemm_fp8(a, sa, w, sw)
        got = f64(Y[r])
        if whole and out == "f32":
            assert np.array_equal(got, want)
            continue
        size = O.gemm_fp8(np.abs(a), sa, np.abs(w), sw)
        tol = (128 * 2.0 ** -23 + (sa.shape[1] + 3) * 2.0 ** -24) * size + HALF[out] * np.abs(want) * (1 + 2.0 ** -7)
        assert np.all(np.abs(got - want) <= tol)


SHAPES = [(1, 1, 16), (1, 128, 128), (3, 7, 16), (16, 64, 256), (17, 200, 144), (64, 256, 512), (65, 129, 272), (100, 1000, 1744),
          (128, 128, 2048), (129, 384, 400), (256, 256, 1024), (300, 520, 640), (512, 96, 128), (5, 2048, 4096), (33, 130, 4112),
          (1, 12288, 512), (200, 72, 7168), (1025, 40, 96), (2, 56, 14336), (260, 1100, 512), (3, 19500, 5120), (2000, 1500, 384), (513, 5000, 1040), (2001, 1501, 384), (1900, 1502, 256), (1800, 2004, 128)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_fp8(dev, M, N, K, out):
    product(dev, M, N, K, out, seed=M + N + K)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_fp8_exact_on_whole_numbers(dev, M, N, K):
    product(dev, M, N, K, "f32", whole=True, seed=M * 3 + N)


@pytest.mark.parametrize("R,M,N,K", [(2, 1, 256, 384), (8, 40, 192, 256), (3, 300, 264, 1024), (16, 130, 128, 144), (8, 600, 512, 512)])
def test_gemm_fp8_ranks(dev, R, M, N, K):
    product(dev, M, N, K, "f32", R=R, whole=True, seed=R)
    product(dev, M, N, K, "bf16", R=R, seed=R)


def random_shapes():
    g = np.random.default_rng(11)
    return [(int(2 ** g.uniform(0, 10.5)), int(2 ** g.uniform(0, 11)), 16 * int(2 ** g.uniform(0, 8)), int(g.integers(1, 4))) for _ in range(40)]


@pytest.mark.parametrize("M,N,K,R", random_shapes())
def test_gemm_fp8_random_shapes(dev, M, N, K, R):
    product(dev, M, N, K, "f32", R=R, whole=True, seed=M + K)


def test_gemm_fp8_repeats_and_keeps_nan_in_its_row(dev):
    g = torch.Generator().manual_seed(1)
    for M in (3, 40, 700):
        N, K = 320, 1152
        A, sA, W, sW = (t.to(dev) for t in operands(g, M, N, K, False))
        A.view(torch.uint8)[1, 7] = 0x7F          # NaN
        sA[2, 3] = float("inf")
        d = B.fo_gemm_fp8_desc(N, K, out_dtype="f32")
        ws = torch.empty(B.fo_gemm_fp8_workspace(d, M), dtype=torch.uint8, device=dev)
        B.fo_ops_workspace_init(ws)
        runs = []
        for _ in range(3):
            Y = torch.zeros(M, N, device=dev)
            B.fo_gemm_fp8(d, M, [A], [sA], [W], [sW], [Y], ws)
            runs.append(Y)
        assert B.fo_ops_status_query(ws)[0] == 0
        assert all(torch.equal(runs[0].view(torch.int32), y.view(torch.int32)) for y in runs[1:])
        got = f64(runs[0])
        assert np.all(np.isnan(got[1])) and not np.any(np.isfinite(got[2]))
        assert np.all(np.isfinite(np.delete(got, (1, 2), axis=0)))


def test_gemm_fp8_input_gradient_with_the_transposed_weight(dev):
    # dX = dY W: dY in 8 bits, the weight's transposed copy. Against the fp64 product of the real values that the 8 bits stand for.
    g = torch.Generator().manual_seed(2)
    M, N, K = 96, 256, 384
    w = (0.02 * torch.randn(N, K, generator=g)).to(torch.bfloat16).to(dev)
    dy = torch.randn(M, N, generator=g).to(torch.bfloat16).to(dev)
    e = lambda *s: torch.empty(s, dtype=E4M3, device=dev)  # noqa: E731
    q, s, qt, st = e(N, K), torch.empty(2, 3, device=dev), e(K, N), torch.empty(3, 2, device=dev)
    B.fo_quant_fp8(N, K, [w], [q], [s], [qt], [st], block_rows=128)
    dq, ds = e(M, N), torch.empty(M, 2, device=dev)
    B.fo_quant_fp8(M, N, [dy], [dq], [ds])
    dx = torch.empty(M, K, device=dev)
    d = B.fo_gemm_fp8_desc(K, N, out_dtype="f32")
    ws = torch.empty(B.fo_gemm_fp8_workspace(d, M), dtype=torch.uint8, device=dev)
    B.fo_ops_workspace_init(ws)
    B.fo_gemm_fp8(d, M, [dq], [ds], [qt], [st], [dx], ws)
    real_dy, real_w = f64(dq) * O.spread(f64(ds), (M, N), 1), f64(q) * O.spread(f64(s), (N, K), 128)
    size = np.abs(real_dy) @ np.abs(real_w)
    assert np.all(np.abs(f64(dx) - real_dy @ real_w) <= (128 * 2.0 ** -23 + 5 * 2.0 ** -24) * size + 2.0 ** -24 * np.abs(real_dy @ real_w))


# Sizes for which tiles of 128 columns are chosen (few of 256, or narrow outputs of many rows): whole and ragged tiles,
# rows of Y that start on 16, 8, 4 and 2 bytes, reductions shorter and longer than the ring.
HALF_TILES = [(1, 512, 4096, 1024), (1, 430, 4100, 272), (2, 511, 1998, 1296), (1, 513, 2051, 2000), (8, 931, 248, 512),
              (4, 3000, 63, 1040), (8, 3000, 97, 640), (2, 3000, 130, 336)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("R,M,N,K", HALF_TILES)
def test_gemm_fp8_tiles_of_128_columns(dev, R, M, N, K, whole, out):
    product(dev, M, N, K, out, R=R, whole=whole, seed=M + N)


# A size for each number of A's rows on a tile (16, 32, 64) and CTAs that share a reduction (1 to 8), as chosen; odd
# outputs, reductions that no number of CTAs divides.
SHARES = [(3, 1, 1945, 2000), (3, 1, 1555, 1376), (3, 1, 932, 1312), (1, 1, 33, 1056), (1, 1, 33, 1440), (1, 1, 32, 1584), (1, 1, 35, 912),
          (3, 49, 3697, 32), (3, 772, 35, 2960), (3, 942, 33, 1840), (1, 1057, 37, 2480), (1, 765, 37, 2080), (3, 194, 33, 4240),
          (2, 476, 33, 3280), (1, 891, 33, 2016), (3, 1538, 32, 4928), (2, 1370, 33, 3184), (1, 1983, 33, 3664), (1, 1785, 35, 4112),
          (1, 1296, 32, 6352), (1, 1824, 67, 2624), (2, 921, 35, 3600), (2, 60, 250, 9008), (1, 128, 4096, 4096)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("R,M,N,K", SHARES)
def test_gemm_fp8_shares_of_the_reduction(dev, R, M, N, K, out):
    product(dev, M, N, K, out, R=R, seed=M + N + K)
