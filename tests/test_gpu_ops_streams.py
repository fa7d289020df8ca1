"""The operators between the residual stream and the attention on streams that are not current, on
several at once and from several threads, and the block's way back replayed from a CUDA graph."""
import threading

import pytest
import torch

from ag_gemm_gb300 import binding as B
from ag_gemm_gb300.layer import Fp8AttentionBlock, LayerShape

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def make(dev, R=2, T=1024, H=1024, seed=0):
    g = torch.Generator().manual_seed(seed)
    width = H // R
    draw = lambda *s, k=1.0: (k * torch.randn(*s, generator=g)).to(BF).to(dev)  # noqa: E731
    block = Fp8AttentionBlock(LayerShape(R=R, T=T, H=H, F=H), device=dev)
    block.set_weights(1 + draw(H, k=0.1), [draw(3 * width, H, k=0.05) for _ in range(R)],
                      [draw(width, H, k=0.02) for _ in range(R)])
    x, res = draw(T, H), draw(T, H)
    grads = [[draw(T, width, k=0.1) for _ in range(R)] for _ in range(3)]
    return block, x, res, torch.arange(T, device=dev), grads, draw(T, H, k=0.1)


def busy(dev, stream):
    """Work of some tens of milliseconds on the stream: what is not ordered behind it runs first."""
    with torch.cuda.stream(stream):
        a = torch.ones(8192, 8192, dtype=BF, device=dev)
        for _ in range(30):
            a @ a


def poison(block):
    torch.cuda.synchronize()
    for t in block.d_qkv + block.dn_part + [block.dn_whole, block.dx, block.dweight, block.h, block.rstd]:
        t.fill_(float("nan"))
    block.n8.view(torch.uint8).fill_(0x7F)
    torch.cuda.synchronize()


def results(block):
    return [t.clone() for t in block.Q + block.K + block.V + [block.h, block.rstd, block.dn_whole, block.dx, block.dweight]]


@pytest.mark.parametrize("how", ["stream", "handle", "default"])
def test_block_on_a_stream_that_is_not_current(dev, how):
    """Behind a long wait on that stream, over poisoned buffers: what is not ordered behind the wait reads the poison."""
    block, x, res, pos, grads, dh = make(dev, seed=len(how))
    block.forward(x, res, pos)
    block.backward(*grads, dh, pos)
    torch.cuda.synchronize()
    want = results(block)
    assert all(torch.isfinite(t.float()).all() for t in want)
    stream = torch.cuda.default_stream() if how == "default" else torch.cuda.Stream()
    s = stream if how == "stream" else stream.cuda_stream
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(2):
            poison(block)
            busy(dev, stream)
            block.forward(x, res, pos, stream=s)
            dx, dweight = block.backward(*grads, dh, pos, stream=s)
            # Allocations of the current stream meanwhile, in the place of whatever the block gave back to it.
            others = [torch.full((block.s.T, block.s.H), float("nan"), dtype=BF, device=dev) for _ in range(4)]
            torch.cuda.synchronize()
            assert block.status() == [0, 0] and len(others) == 4
            assert dx is block.dx and dweight is block.dweight
            assert all(torch.equal(a, b) for a, b in zip(results(block), want))


def test_block_status_waits_for_the_stream_it_is_asked_on(dev):
    block, x, res, pos, grads, dh = make(dev, T=256)
    stream = torch.cuda.Stream()
    for s in (stream, stream.cuda_stream):
        torch.cuda.synchronize()
        busy(dev, stream)
        block.forward(x, res, pos, stream=s)
        assert block.status(stream=s) == [0, 0]
        assert stream.query()


def test_block_is_ready_for_any_stream_once_it_is_made(dev):
    # The workspaces are zeroed on the stream that is current: a first call on another one finds them zeroed.
    first = torch.cuda.Stream()
    busy(dev, first)
    with torch.cuda.stream(first):
        block = Fp8AttentionBlock(LayerShape(R=2, T=256, H=256, F=256), device=dev)
    assert first.query()


def test_block_backward_from_a_graph(dev):
    block, x, res, pos, grads, dh = make(dev, R=4, seed=3)
    block.forward(x, res, pos)
    block.backward(*grads, dh, pos)
    torch.cuda.synchronize()
    want = results(block)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        block.forward(x, res, pos)
        block.backward(*grads, dh, pos)
    for _ in range(2):
        poison(block)
        graph.replay()
        torch.cuda.synchronize()
        assert block.status() == [0, 0]
        assert all(torch.equal(a, b) for a, b in zip(results(block), want))
    # Other gradients in the same place are read afresh.
    grads[0][0].neg_()
    graph.replay()
    torch.cuda.synchronize()
    again = results(block)
    assert not torch.equal(again[-2], want[-2])
    block.backward(*grads, dh, pos)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(results(block), again))


def test_norms_quantiser_and_rotary_on_streams_at_once(dev):
    """Calls with their own outputs and workspaces may overlap: the results are those of calls one after another."""
    g = torch.Generator().manual_seed(4)
    jobs = []
    for rows, H in ((3000, 4096), (700, 8184), (2500, 1357), (4, 4096)):
        x, res, dy = (torch.randn(rows, H, generator=g).to(BF).to(dev) for _ in range(3))
        w, d = torch.ones(H, dtype=BF, device=dev), B.fo_norm_desc(H)
        new = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device=dev)  # noqa: E731
        h, q, sc, r, dx, dw = new(rows, H, t=BF), new(rows, H), new(rows, -(-H // 128), t=torch.float32), \
            new(rows, t=torch.float32), new(rows, H, t=BF), new(H, t=torch.float32)
        q2, sc2, turned = new(rows, H), new(rows, -(-H // 128), t=torch.float32), new(rows, H, t=BF)
        ws = torch.empty(B.fo_rmsnorm_bwd_workspace(d, rows), dtype=torch.uint8, device=dev)
        rope = B.fo_rope_desc(64, H // 64)
        width = H // 64 * 64

        def go(stream, a=(rows, H, x, res, dy, w, d, h, q, sc, r, dx, dw, q2, sc2, turned, ws, rope, width)):
            rows, H, x, res, dy, w, d, h, q, sc, r, dx, dw, q2, sc2, turned, ws, rope, width = a
            B.fo_rmsnorm(d, rows, [x], [res], w, [h], None, [q], [sc], [r], stream=stream)
            B.fo_rmsnorm_bwd(d, rows, [dy], [res], [h], w, [r], [dx], dw, ws, stream=stream)
            B.fo_quant_fp8(rows, H, [dx], [q2], [sc2], stream=stream)
            B.fo_rope(rope, rows, None, [dx[:, :width]], None, None, [turned[:, :width]], None, None, stream=stream)

        jobs.append((go, [h, q, sc, r, dx, dw, q2, sc2, turned], width, torch.cuda.Stream()))
    torch.cuda.synchronize()
    values = lambda outs, width: outs[:-1] + [outs[-1][:, :width]]  # noqa: E731
    for go, _, _, stream in jobs:
        go(stream)
        torch.cuda.synchronize()
    want = [[t.clone() for t in values(outs, width)] for _, outs, width, _ in jobs]
    for _, outs, _, _ in jobs:
        for t in outs:
            t.view(torch.uint8).fill_(0x7F)
    torch.cuda.synchronize()
    for _ in range(20):
        for go, _, _, stream in jobs:
            go(stream)
    torch.cuda.synchronize()
    for (_, outs, width, _), ref in zip(jobs, want):
        assert all(torch.equal(a, b) for a, b in zip(values(outs, width), ref))


@pytest.mark.parametrize("dtype,widths", [("bf16", (4352, 8184)), ("bf16", (8448, 16376)), ("f32", (2176, 4092))])
def test_norm_backward_from_two_threads(dev, dtype, widths):
    """Two widths that one kernel serves with different amounts of shared memory, from two threads: no call may change
    what the other's launch is allowed."""
    T = {"bf16": BF, "f32": torch.float32}[dtype]
    errors, rows = [], 5

    def work(H):
        try:
            dy, h, w, r = (torch.ones(s, dtype=t, device=dev) for s, t in (((rows, H), T), ((rows, H), T), ((H,), T), ((rows,), torch.float32)))
            dx, dw, d = torch.empty_like(dy), torch.empty(H, device=dev), B.fo_norm_desc(H, dtype=dtype)
            ws = torch.empty(B.fo_rmsnorm_bwd_workspace(d, rows), dtype=torch.uint8, device=dev)
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            for i in range(6000):
                B.fo_rmsnorm_bwd(d, rows, [dy], None, [h], w, [r], [dx], dw, ws, stream=stream)
                if i % 500 == 499:
                    stream.synchronize()
            # Each row's gradient is 1 - 1 * mean(1); the weight's the number of rows.
            assert torch.count_nonzero(dx).item() == 0 and (dw == rows).all()
        except Exception as e:   # noqa: BLE001 (told by the test)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(H,)) for H in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
