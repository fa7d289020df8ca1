"""The operators on tensors of more than 2^31 values: rows that repeat give results that repeat, to the last of them. And
replayed from graphs in which a call follows a memset or joins two streams."""
import pytest
import torch

from ag_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32
FEW = 7


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def new(dev, *s, dtype=F32):
    return torch.zeros(s, dtype=dtype, device=dev)


def repeats(many, few):
    """Every run of len(few) rows of `many` is `few`, compared a slice at a time."""
    n = few.shape[0]
    part = 4096 * n
    return all(torch.equal(p, few.repeat(p.shape[0] // n, 1)) for p in many.split(part))


@pytest.mark.parametrize("H", [4096, 4095])
def test_norm_and_row_quantiser(dev, H):
    g = torch.Generator().manual_seed(H)
    few = [(torch.randn(FEW, H, generator=g)).to(BF).to(dev) for _ in range(2)]
    w, d, groups = torch.rand(H, generator=g).to(BF).to(dev), B.fo_norm_desc(H), -(-H // 128)

    def run(x, dy):
        n = x.shape[0]
        y, q, s, r = new(dev, n, H, dtype=BF), new(dev, n, H, dtype=U8), new(dev, n, groups), new(dev, n)
        B.fo_rmsnorm(d, n, [x], None, w, None, [y], [q], [s], [r])
        dx, dw = new(dev, n, H, dtype=BF), new(dev, H)
        B.fo_rmsnorm_bwd(d, n, [dy], None, [x], w, [r], [dx], dw, new(dev, B.fo_rmsnorm_bwd_workspace(d, n), dtype=U8))
        q2, s2 = new(dev, n, H, dtype=U8), new(dev, n, groups)
        B.fo_quant_fp8(n, H, [x], [q2], [s2])
        return y, q, s, r[:, None], dx, q2, s2

    times = -(-(1 << 31) // (FEW * H)) + 30
    want = run(*few)
    got = run(*(t.repeat(times, 1) for t in few))
    assert got[0].numel() > 1 << 31
    assert all(repeats(m, f) and torch.count_nonzero(f) for m, f in zip(got, want))


@pytest.mark.parametrize("cols", [4096, 4098])
def test_block_quantiser(dev, cols):
    g = torch.Generator().manual_seed(cols)
    few = torch.randn(128, cols, generator=g).to(BF).to(dev)
    times = -(-(1 << 31) // (128 * cols)) + 3
    rows, across = 128 * times, -(-cols // 128)
    x = few.repeat(times, 1)
    q, s, qt, st = new(dev, rows, cols, dtype=U8), new(dev, times, across), new(dev, cols, rows, dtype=U8), new(dev, across, times)
    B.fo_quant_fp8(rows, cols, [x], [q], [s], [qt], [st], block_rows=128)
    q1, s1 = new(dev, 128, cols, dtype=U8), new(dev, 1, across)
    B.fo_quant_fp8(128, cols, [few], [q1], [s1], block_rows=128)
    assert q.numel() > 1 << 31 and repeats(q, q1) and repeats(s, s1) and torch.count_nonzero(q1)
    assert torch.equal(st, s.t()) and all(torch.equal(a, b) for a, b in zip(qt.split(256), q.t().split(256)))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_positions(dev, layout):
    heads, D = 20, 128
    width = heads * D
    few = torch.randn(FEW, 3 * width, generator=torch.Generator().manual_seed(1)).to(BF).to(dev)
    times = -(-(1 << 31) // (FEW * 3 * width)) + 30
    pos = torch.tensor([0, 5, -3, 100000, 1 << 40, 77, 1], device=dev)

    def run(x, p):
        outs = [new(dev, x.shape[0], width, dtype=BF) for _ in range(3)]
        B.fo_rope(B.fo_rope_desc(D, heads, heads, heads, layout=layout), x.shape[0], p, *[[t] for t in x.split(width, dim=1)], *[[o] for o in outs])
        return outs

    want, x = run(few, pos), few.repeat(times, 1)
    assert x.numel() > 1 << 31
    assert all(repeats(m, f) and torch.count_nonzero(f) for m, f in zip(run(x, pos.repeat(times)), want))


@pytest.mark.parametrize("N", [32768, 32770, 32769])
def test_product_with_a_large_output(dev, N):
    g = torch.Generator().manual_seed(N)
    K, times = 128, -(-(1 << 31) // (FEW * N)) + 30
    A, W = (torch.randint(-4, 5, s, generator=g).float().to(torch.float8_e4m3fn).to(dev) for s in ((FEW, K), (N, K)))
    sA = (torch.rand(FEW, 1, generator=g) + 0.5).to(dev)
    d, sW = B.fo_gemm_fp8_desc(N, K), new(dev, -(-N // 128), 1) + 0.25
    A8, many, Y = A.view(U8).repeat(times, 1), FEW * times, new(dev, FEW * times, N, dtype=BF)
    ws = new(dev, B.fo_gemm_fp8_workspace(d, many), dtype=U8)
    B.fo_gemm_fp8(d, many, [A8], [sA.repeat(times, 1)], [W], [sW], [Y], ws)
    assert B.fo_ops_status_query(ws)[0] == 0 and Y.numel() > 1 << 31
    want = ((A.float() @ W.float().t()) * (sA * 0.25)).to(BF)   # whole numbers below 2^11, one rounding by the scale, one to bf16
    assert repeats(Y, want)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_product_with_a_large_weight(dev, M):
    g = torch.Generator().manual_seed(M)
    K, base = 4096, 512
    N = (1 << 31) // K + 4 * base
    A, W = (torch.randint(-4, 5, s, generator=g).float().to(torch.float8_e4m3fn).to(dev) for s in ((M, K), (base, K)))
    d, ws = B.fo_gemm_fp8_desc(N, K, out_dtype="f32"), None
    ws = new(dev, B.fo_gemm_fp8_workspace(d, M), dtype=U8)
    Y, big = new(dev, M, N), W.view(U8).repeat(N // base, 1)
    assert big.numel() > 1 << 31
    B.fo_gemm_fp8(d, M, [A], [new(dev, M, K // 128) + 1], [big], [new(dev, N // 128, K // 128) + 1], [Y], ws)
    assert B.fo_ops_status_query(ws)[0] == 0
    want = A.double() @ W.double().t()
    assert all(torch.equal(p.double(), want) for p in Y.split(base, dim=1))


def test_graph_with_a_memset_before_and_streams_that_join(dev):
    g = torch.Generator().manual_seed(2)
    rows, H = 300, 1024
    x, res = (torch.randn(rows, H, generator=g).to(BF).to(dev) for _ in range(2))
    w, d, p = torch.ones(H, dtype=BF, device=dev), B.fo_norm_desc(H), B.fo_gemm_fp8_desc(H, H, out_dtype="f32")
    h, q, s, r = new(dev, rows, H, dtype=BF), new(dev, rows, H, dtype=U8), new(dev, rows, 8), new(dev, rows)
    W8, sW, y = new(dev, H, H, dtype=U8), new(dev, 8, 8), new(dev, rows, H)
    weight = torch.randn(H, H, generator=g).to(BF).to(dev)
    ws = new(dev, B.fo_gemm_fp8_workspace(p, rows), dtype=U8)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        B.fo_ops_workspace_init(ws)                                          # a memset
        B.fo_rmsnorm(d, rows, [x], [res], w, [h], None, [q], [s], [r])
        side.wait_stream(main)
        B.fo_quant_fp8(H, H, [weight], [W8], [sW], block_rows=128, stream=side)
        B.fo_rmsnorm(d, rows, [res], [x], w, [h], None, [q], [s], [r])
        main.wait_stream(side)
        B.fo_gemm_fp8(p, rows, [q], [s], [W8], [sW], [y], ws)                # after both streams' kernels

    outs = (h, q, s, r, W8, sW, y)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.count_nonzero(a) for a, b in zip(outs, want))
    assert B.fo_ops_status_query(ws)[0] == 0
