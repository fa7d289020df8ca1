"""The operators between the residual stream and the attention as they are used: a block of the layer from the
residual stream to the reduce-scattered output and the gradients' way back, on another stream, and replayed from a
CUDA graph. Each stage is held to the oracle on the inputs that the GPU gave it, with the tolerances of the operators'
own tests (test_gpu_norm_quant.py, test_gpu_gemm_fp8.py, test_gpu_rope.py, test_gpu_attn.py)."""
import numpy as np
import pytest
import torch

import oracle
from ag_gemm_gb300.layer import Fp8AttentionBlock, LayerShape
from oracle import layer_ops as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E4M3_STEP = 2.0 ** -4


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


def make(dev, R=2, T=512, H=512, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    block = Fp8AttentionBlock(LayerShape(R=R, T=T, H=H, F=H), device=dev, **kw)
    bf = torch.bfloat16
    W = [(0.05 * torch.randn(3 * H // R, H, generator=g)).to(bf).to(dev) for _ in range(R)]
    Wo = [(0.02 * torch.randn(H // R, H, generator=g)).to(bf).to(dev) for _ in range(R)]
    weight = (1 + 0.1 * torch.randn(H, generator=g)).to(bf).to(dev)
    block.set_weights(weight, W, Wo)
    x, res = (torch.randn(T, H, generator=g).to(bf).to(dev) for _ in range(2))
    return block, W, x, res, g


def check_forward(block, x, res, positions, W):
    T, H, R = block.s.T, block.s.H, block.s.R
    width = H // R
    s, n, r = O.rmsnorm(f64(x), f64(res), f64(block.weight), 1e-6)
    assert np.all(np.abs(f64(block.h) - s) <= (2.0 ** -8 + U) * np.abs(s))
    assert np.all(np.abs(f64(block.rstd) - r) <= 44 * U * r)
    each = O.spread(f64(block.n_scale), n.shape, 1)
    assert np.all(np.abs(f64(block.n8) * each - n) <= E4M3_STEP * np.abs(n) * (1 + 1e-4) + 2.0 ** -10 * each)
    f, factor = O.rope_frequencies(128, 10000.0)
    for k in range(R):
        w = f64(block.Wq[k]) * O.spread(f64(block.Wq_scale[k]), W[k].shape, 128)
        assert np.all(np.abs(w - f64(W[k])) <= E4M3_STEP * np.abs(f64(W[k])) * (1 + 1e-5) + 2.0 ** -10 * O.spread(f64(block.Wq_scale[k]), W[k].shape, 128))
        a = f64(block.n8) * each
        y, size = a @ w.T, np.abs(a) @ np.abs(w).T
        assert np.all(np.abs(f64(block.y_qkv[k]) - y) <= (128 * 2.0 ** -23 + (H // 128 + 3) * U) * size + 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -7))
        parts = np.split(f64(block.y_qkv[k]), 3, axis=1)
        for got, part in ((block.Q[k], parts[0]), (block.K[k], parts[1])):
            want = O.rope(part, positions, f, factor, 128, "half")
            v = np.abs(part.reshape(T, -1, 2, 64)).sum(axis=2, keepdims=True).repeat(2, axis=2).reshape(T, -1)
            assert np.all(np.abs(f64(got) - want) <= 8 * U * v + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7))
        assert np.array_equal(f64(block.V[k]), parts[2])
        q, kk, v = f64(block.Q[k]), f64(block.K[k]), f64(block.V[k])
        ref = oracle.round_bf16(oracle.attention(q, kk, v, block.heads, True))
        absw = oracle.attention(q, kk, np.abs(v), block.heads, True)
        assert np.all(np.abs(f64(block.O[k]) - ref) <= 1.25 * (2.0 ** -8 * absw + 2.0 ** -7 * np.abs(ref)))
    proj = oracle.gemm_rs([f64(o) for o in block.O], [f64(w) for w in block.Wo])
    for d in range(R):
        fro, mx, _ = oracle.rel_errors(f64(block.y[d]), oracle.round_bf16(proj[d]))
        assert fro <= 1e-3 and mx <= 2e-2


def test_block_forward(dev):
    block, W, x, res, _ = make(dev)
    pos = torch.arange(block.s.T, device=dev)
    block.forward(x, res, pos)
    assert block.status() == [0, 0]
    check_forward(block, x, res, pos.cpu().numpy().astype(np.float64), W)


def test_block_backward(dev):
    block, W, x, res, g = make(dev, seed=1)
    T, H, R = block.s.T, block.s.H, block.s.R
    width = H // R
    pos = torch.arange(T, device=dev) + 5
    block.forward(x, res, pos)
    dQ, dK, dV = ([(0.1 * torch.randn(T, width, generator=g)).to(torch.bfloat16).to(dev) for _ in range(R)] for _ in range(3))
    dh = (0.1 * torch.randn(T, H, generator=g)).to(torch.bfloat16).to(dev)
    dx, dweight = block.backward(dQ, dK, dV, dh, pos)
    assert block.status() == [0, 0]
    f, factor = O.rope_frequencies(128, 10000.0)
    p = pos.cpu().numpy().astype(np.float64)
    dn = np.zeros((T, H))
    size = np.zeros((T, H))
    for k in range(R):
        back = np.concatenate([O.rope(f64(d[k]), p, f, factor, 128, "half", inverse=True) for d in (dQ, dK)] + [f64(dV[k])], axis=1)
        got = f64(block.d_qkv[k])
        assert np.all(np.abs(got - back) <= 2.0 ** -8 * np.abs(back) * (1 + 2.0 ** -7) + 16 * U * np.max(np.abs(back)))
        a = f64(block.d8[k]) * O.spread(f64(block.d_scale[k]), back.shape, 1)
        w = f64(block.Wt[k]) * O.spread(f64(block.Wt_scale[k]), (H, 3 * width), 128)
        assert np.array_equal(f64(block.Wt[k]), f64(block.Wq[k]).T)
        dn += a @ w.T
        size += np.abs(a) @ np.abs(w).T
    got = f64(torch.cat(block.dn))
    assert np.all(np.abs(got - dn) <= (128 * 2.0 ** -23 + (3 * width // 128 + 3 + R) * U) * size)
    dy = f64(torch.cat(block.dn).to(torch.bfloat16))
    want_x, want_w = O.rmsnorm_bwd(dy, f64(dh), f64(block.h), f64(block.weight), f64(block.rstd))
    r = f64(block.rstd)[:, None]
    u = np.abs(dy * f64(block.weight))
    b = np.abs(f64(block.h)) * r ** 3 * np.mean(u * np.abs(f64(block.h)), axis=1)[:, None]
    assert np.all(np.abs(f64(dx) - want_x) <= 2.0 ** -8 * np.abs(want_x) * (1 + 2.0 ** -7) + 4 * U * (r * u + np.abs(f64(dh))) + 90 * U * b)
    assert np.all(np.abs(f64(dweight) - want_w) <= (T + 4) * U * np.sum(np.abs(dy * f64(block.h) * r), axis=0))


def test_block_from_a_graph_on_another_stream(dev):
    block, W, x, res, _ = make(dev, R=4, T=1024, H=1024, seed=2)
    pos = torch.arange(block.s.T, device=dev)
    block.forward(x, res, pos)
    first = [t.clone() for t in block.y + block.Q + [block.n8.view(torch.uint8), block.h]]
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        block.forward(x, res, pos)                      # eagerly on this stream first
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            block.forward(x, res, pos)
    for t in block.y + block.Q + block.K + block.V + block.y_qkv:
        t.fill_(float("nan"))
    block.n8.view(torch.uint8).fill_(0x7F)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    now = block.y + block.Q + [block.n8.view(torch.uint8), block.h]
    for i, (a, b) in enumerate(zip(first, now)):
        if i < 4:   # the projection's partials are added as they arrive
            fro, mx, _ = oracle.rel_errors(f64(b), f64(a))
            assert fro <= 1e-3 and mx <= 2e-2
        else:
            assert torch.equal(a, b)
    # Other inputs in the same place: the graph reads them afresh.
    x.copy_(torch.randn(x.shape).to(torch.bfloat16))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert block.status() == [0, 0]
    assert not torch.equal(first[-1], block.h)
    s, n, r = O.rmsnorm(f64(x), f64(res), f64(block.weight), 1e-6)
    assert np.all(np.abs(f64(block.rstd) - r) <= 44 * U * r)


def test_product_and_norm_on_two_streams_at_once(dev):
    # Calls with their own workspaces may overlap: results are those of calls one after another.
    from ag_gemm_gb300 import binding as B
    g = torch.Generator().manual_seed(3)
    e4m3 = torch.float8_e4m3fn
    jobs = []
    for i, (M, N, K) in enumerate([(700, 1024, 2048), (4, 4096, 4096), (64, 2048, 1024), (900, 768, 4096)]):
        A, W = (torch.randint(-4, 5, s, generator=g).float().to(e4m3).to(dev) for s in ((M, K), (N, K)))
        sA, sW = torch.ones(M, K // 128, device=dev), torch.ones(N // 128, K // 128, device=dev)
        d = B.fo_gemm_fp8_desc(N, K, out_dtype="f32")
        ws = torch.empty(B.fo_gemm_fp8_workspace(d, M), dtype=torch.uint8, device=dev)
        B.fo_ops_workspace_init(ws)
        jobs.append((d, M, [A], [sA], [W], [sW], [torch.zeros(M, N, device=dev)], ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for *args, stream in jobs:
            B.fo_gemm_fp8(*args, stream)
    torch.cuda.synchronize()
    for d, M, A, sA, W, sW, Y, ws, stream in jobs:
        assert B.fo_ops_status_query(ws)[0] == 0
        assert np.array_equal(f64(Y[0]), f64(A[0]) @ f64(W[0]).T)


def test_addresses_and_tensors_make_the_same_call(dev):
    # Tensors are checked and passed on by the native marshalling module, raw addresses by the Python binding.
    from ag_gemm_gb300 import binding as B
    e4m3 = torch.float8_e4m3fn
    rows, H = 5, 640
    x, res = (torch.randn(rows, H).to(torch.bfloat16).to(dev) for _ in range(2))
    w = torch.rand(H).to(torch.bfloat16).to(dev)
    got = []
    for raw in (False, True):
        a = (lambda t: t.data_ptr()) if raw else (lambda t: t)
        h, q = torch.zeros_like(x), torch.zeros(rows, H, dtype=e4m3, device=dev)
        s, r = torch.zeros(rows, 5, device=dev), torch.zeros(rows, device=dev)
        B.fo_rmsnorm(B.fo_norm_desc(H), rows, [a(x)], [a(res)], a(w), [a(h)], None, [a(q)], [a(s)], [a(r)])
        dx, dw = torch.zeros_like(x), torch.zeros(H, device=dev)
        ws = torch.zeros(B.fo_rmsnorm_bwd_workspace(B.fo_norm_desc(H), rows), dtype=torch.uint8, device=dev)
        B.fo_rmsnorm_bwd(B.fo_norm_desc(H), rows, [a(x)], [a(res)], [a(h)], a(w), [a(r)], [a(dx)], a(dw), a(ws))
        wq, wsc = torch.zeros(rows, H, dtype=e4m3, device=dev), torch.zeros(1, 5, device=dev)
        B.fo_quant_fp8(rows, H, [a(x)], [a(wq)], [a(wsc)], block_rows=128, dtype="bf16")
        y, g = torch.zeros(rows, rows, device=dev), B.fo_gemm_fp8_desc(rows, H, out_dtype="f32")
        gws = torch.zeros(B.fo_gemm_fp8_workspace(g, rows), dtype=torch.uint8, device=dev)
        B.fo_gemm_fp8(g, rows, [a(q)], [a(s)], [a(wq)], [a(wsc)], [a(y)], a(gws))
        turned, pos = torch.zeros_like(x), torch.arange(rows, device=dev)
        B.fo_rope(B.fo_rope_desc(128, 5), rows, a(pos), [a(x)], None, None, [a(turned)], None, None)
        got.append([h, q.view(torch.uint8), s, r, dx, dw, wq.view(torch.uint8), wsc, y, turned])
    for u, v in zip(*got):
        assert torch.equal(u, v) and torch.count_nonzero(u)


def test_binding_refuses_small_workspaces_and_wrong_sizes(dev):
    from ag_gemm_gb300 import binding as B
    d = B.fo_norm_desc(256)
    t = torch.zeros(4, 256, dtype=torch.bfloat16, device=dev)
    r = torch.zeros(4, device=dev)
    with pytest.raises(ValueError, match="workspace"):
        B.fo_rmsnorm_bwd(d, 4, [t], None, [t], t[0], [r], [t], torch.zeros(256, device=dev), torch.zeros(16, dtype=torch.uint8, device=dev))
    q, s = torch.zeros(4, 256, dtype=torch.uint8, device=dev), torch.zeros(4, 2, device=dev)
    g = B.fo_gemm_fp8_desc(4, 256)
    with pytest.raises(ValueError, match="workspace"):
        B.fo_gemm_fp8(g, 4, [q], [s], [q], [s[:1]], [t[:, :4].contiguous()], torch.zeros(8, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="values given"):
        B.fo_quant_fp8(4, 256, [t], [q], [s[:, :1].contiguous()])
    with pytest.raises(ValueError, match="contiguous"):
        B.fo_quant_fp8(256, 4, [t.t()], [q], [torch.zeros(256, 1, device=dev)])
    with pytest.raises(ValueError, match="rows of"):
        B.fo_rope(B.fo_rope_desc(128, 2), 4, None, [t[:, :128]], None, None, [t], None, None)


@pytest.mark.parametrize("M,N,K", [(4, 512, 512), (1024, 1024, 512)])
def test_inputs_rewritten_by_the_kernel_before(dev, M, N, K):
    """Kernels may be set up before the one ahead of them has ended: the same buffers, written again by each kernel
    before (8-bit rows, scales, weights with their scales, a norm's weight), are read as they were just written. The
    calls without a wait between them give the very bits that the same calls with waits give."""
    from ag_gemm_gb300 import binding as B
    g = torch.Generator().manual_seed(5)
    n = 8
    X = [(2.0 ** i * torch.randn(M, K, generator=g)).bfloat16().to(dev) for i in range(n)]
    Ws = [(2.0 ** -i * torch.randn(N, K, generator=g)).bfloat16().to(dev) for i in range(n)]
    dY = [torch.randn(M, K, generator=g).bfloat16().to(dev) for i in range(n)]
    u8 = torch.uint8
    q, s = torch.empty(M, K, dtype=u8, device=dev), torch.empty(M, K // 128, device=dev)
    w, sw = torch.empty(N, K, dtype=u8, device=dev), torch.empty(N // 128, K // 128, device=dev)
    gain, rstd, dx = torch.ones(K, device=dev), torch.ones(M, device=dev), torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    product, norm = B.fo_gemm_fp8_desc(N, K, out_dtype="f32"), B.fo_norm_desc(K, dtype="bf16", w_dtype="f32")
    ws = torch.empty(B.fo_gemm_fp8_workspace(product, M), dtype=u8, device=dev)
    B.fo_ops_workspace_init(ws)
    wsn = torch.empty(B.fo_rmsnorm_bwd_workspace(norm, M), dtype=u8, device=dev)

    def run(wait):
        gain.fill_(1.0)
        out = []
        for i in range(n):
            y, y2 = torch.empty(M, N, device=dev), torch.empty(M, K, dtype=torch.bfloat16, device=dev)
            y3 = torch.empty(M, N, device=dev)
            torch.cuda.synchronize()
            calls = [lambda: B.fo_quant_fp8(N, K, [Ws[i]], [w], [sw], block_rows=128),
                     lambda: B.fo_quant_fp8(M, K, [X[i]], [q], [s]),
                     lambda: B.fo_gemm_fp8(product, M, [q], [s], [w], [sw], [y], ws),
                     lambda: B.fo_rmsnorm_bwd(norm, M, [dY[i]], None, [X[i]], gain, [rstd], [dx], gain, wsn),
                     lambda: B.fo_rmsnorm(norm, M, [dx], None, gain, y=[y2], q=[q], scale=[s], rstd=[rstd]),
                     lambda: B.fo_gemm_fp8(product, M, [q], [s], [w], [sw], [y3], ws)]
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
            out += [y, dx.clone(), y2, rstd.clone(), gain.clone(), y3]
            gain.div_(gain.abs().max())
        torch.cuda.synchronize()
        return out

    rstd.fill_(1.0)
    want = run(True)
    for _ in range(3):
        rstd.fill_(1.0)
        got = run(False)
        assert all(torch.isfinite(t.float()).all() for t in want)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert B.fo_ops_status_query(ws)[0] == 0
