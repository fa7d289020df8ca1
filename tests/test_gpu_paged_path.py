"""Serving from a paged cache as it is used: the block's operators one after another (prompts, then tokens one at a time
from a replayed graph), on other streams, two at once, and over caches larger than 32 bits count.

Each stage of the block is held to the oracle's result from what the stage before wrote, with that operator's own bound
(see the operators' tests); the o product and its sum as the QKV product: 128 products of fp32 a block in an order of
its own, one sum over the blocks, one over the ranks.
"""
import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from ag_gemm_gb300.layer import PagedAttentionBlock
from oracle import layer_ops as O
from oracle import paged as P
from test_gpu_paged import BF, E4M3, NAN, U, Cache, f64, first_rows, held_to_the_oracle, turned, whole, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def weights(block, dev, g):
    width = sum(block.widths)
    draw = lambda *s, k=1.0: (k * torch.randn(*s, generator=g)).to(BF).to(dev)  # noqa: E731
    W = [draw(width, block.H, k=0.05) for _ in range(block.R)]
    Wo = [draw(block.H, block.width, k=0.02) for _ in range(block.R)]
    block.set_weights(1 + draw(block.H, k=0.1), W, Wo)
    return W, Wo


def wide(q, scale, up=1):
    return f64(q) * O.spread(f64(scale), q.shape, up)


def held(block, r, b, length, page):
    """What rank r's cache holds of sequence b: keys, values [length, heads_k, D] in fp64."""
    pg, slot = P.places(block.table[b].cpu().numpy(), length, page)
    out = []
    for c, s in ((block.k[r], block.k_scale and block.k_scale[r]), (block.v[r], block.v_scale and block.v_scale[r])):
        x = f64(c[torch.from_numpy(pg.astype(np.int64)).to(c.device)].float())[np.arange(length), :, slot]
        if s is not None:
            x = x * f64(s[torch.from_numpy(pg.astype(np.int64)).to(c.device)])[np.arange(length), :, slot][..., None]
        out.append(x)
    return out


def check(block, x, residual, lengths, new, before):
    """A call's stages; `before`: what the cache held, [r][b] of (keys, values)."""
    d, H, R = block.paged, block.H, block.R
    assert block.status() == [0, 0]
    s, n, _ = O.rmsnorm(f64(x), None if residual is None else f64(residual), f64(block.weight), 1e-6)
    assert np.all(np.abs(f64(block.h) - s) <= (2.0 ** -8 + U) * np.abs(s))
    each = O.spread(f64(block.n_scale), n.shape, 1)
    assert np.all(np.abs(f64(block.n8) * each - n) <= 2.0 ** -4 * np.abs(n) * (1 + 1e-4) + 2.0 ** -10 * each)
    rows = [(b, L - m + i) for b, (L, m) in enumerate(zip(lengths, new)) for i in range(m)]
    used, pos = len(rows), np.array([p for _, p in rows], dtype=np.float64)
    after = []
    for r in range(R):
        a, w = wide(block.n8, block.n_scale), wide(block.Wq[r], block.Wq_scale[r], 128)
        y, size = a @ w.T, np.abs(a) @ np.abs(w).T
        assert np.all(np.abs(f64(block.y_qkv[r]) - y) <= (128 * 2.0 ** -23 + (H // 128 + 3) * U) * size + 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -7))
        q, k, v = np.split(f64(block.y_qkv[r])[:used], np.cumsum(block.widths)[:2], axis=1)
        want, off = turned(q, pos, d, block.rope)
        assert np.all(np.abs(f64(block.Q[r])[:used] - want) <= off + 2.0 ** -8 * (np.abs(want) + off))
        after.append([held(block, r, b, L, d.page) for b, L in enumerate(lengths)])
        want, off = turned(k, pos, d, block.rope)
        at = 0
        for b, (L, m) in enumerate(zip(lengths, new)):
            for j, (x_new, x_off) in enumerate(((want, off), (v, np.zeros_like(v)))):
                got, kept = after[r][b][j], before[r][b][j]
                assert np.array_equal(got[:L - m], kept[:L - m])          # (older tokens)
                mine, w_, o_ = got[L - m:], x_new[at:at + m].reshape(m, d.heads_k, d.head_dim), x_off[at:at + m].reshape(m, d.heads_k, d.head_dim)
                if d.cache_dtype == 0:
                    assert np.all(np.abs(mine - w_) <= o_ + 2.0 ** -8 * (np.abs(w_) + o_))
                else:
                    scale = np.maximum(np.abs(w_).max(axis=2, keepdims=True) / 448, 2.0 ** -126) if m else 0.0
                    assert np.all(np.abs(mine - w_) <= o_ + 2.0 ** -4 * (np.abs(w_) + o_) * (1 + 1e-4) + 2.0 ** -10 * scale * (1 + 1e-4))
            at += m
    whole_o = [f64(o) for o in block.O]
    cache = type("", (), dict(d=d, lengths=lengths, new=new, k=[[x[0] for x in a] for a in after], v=[[x[1] for x in a] for a in after]))
    held_to_the_oracle(cache, [f64(q) for q in block.Q], whole_o, None)
    total, size = 0, 0
    for r in range(R):
        o = wide(block.o8[r], block.o_scale[r])
        each = O.spread(f64(block.o_scale[r]), o.shape, 1)
        assert np.all(np.abs(o - whole_o[r]) <= 2.0 ** -4 * np.abs(whole_o[r]) * (1 + 1e-5) + 2.0 ** -10 * each)
        w = wide(block.Wo[r], block.Wo_scale[r], 128)
        total, size = total + o @ w.T, size + np.abs(o) @ np.abs(w).T
    assert np.all(np.abs(f64(block.y_whole) - total) <= (128 * 2.0 ** -23 + (-(-block.width // 128) + 3 + R) * U) * size)
    return after


CASES = [  # R, H, heads_q, heads_k, D, page, cache, window, sinks
    (2, 512, 8, 2, 128, 16, "e4m3", 0, 0),
    (3, 192, 4, 4, 64, 32, "bf16", 24, 4),
    (1, 256, 20, 1, 128, 64, "e4m3", 40, 0),
]


@pytest.mark.parametrize("case", CASES)
def test_prompts_then_tokens(dev, case):
    R, H, hq, hk, D, page, kept, window, sinks = case
    g = torch.Generator().manual_seed(11)
    prompts, pages = [70, 1, 33], 24
    common = dict(seqs=3, pages=pages, cols=8, R=R, head_dim=D, page=page, cache=kept, window=window, sinks=sinks, device=dev)
    first = PagedAttentionBlock(H, hq, hk, rows=108, max_new=80, **common)
    weights(first, dev, g)
    token = PagedAttentionBlock(H, hq, hk, rows=6, like=first, **common)
    for block in (first, token):
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(1))
        block.table.copy_(order[:24].view(3, 8))
    nothing = [[held(first, r, b, 0, page) for b in range(3)] for r in range(R)]
    x, res = (torch.randn(108, H, generator=g).to(BF).to(dev) for _ in range(2))
    # the first call has the prompts' beginnings, the second their rest
    lengths, before = [0, 0, 0], nothing
    for new in ([30, 0, 33], [40, 1, 0]):
        lengths = [a + b for a, b in zip(lengths, new)]
        first.lengths.copy_(whole(lengths, dev)), first.starts.copy_(whole(first_rows(new), dev))
        first.forward(x, res)
        before = check(first, x, res, lengths, new, before)
    assert lengths == prompts
    # tokens: one captured step, replayed with other inputs, lengths and a sequence that ends
    xt = torch.zeros(6, H, dtype=BF, device=dev)
    token.forward(xt)                                       # (sequences that are not there: loads the kernels)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token.forward(xt)
    for step in range(4):
        new = [1, 1, 0 if step == 2 else 1]
        lengths = [a + b for a, b in zip(lengths, new)]
        token.lengths.copy_(whole([n if m else 0 for n, m in zip(lengths, new)], dev))
        xt.copy_(torch.randn(6, H, generator=g).to(BF))
        graph.replay()
        if new[2]:
            before = check(token, xt, None, lengths, new, before)
        else:
            assert token.status() == [0, 0] and all((o[2] == 0).all() for o in token.O)
            before = [[held(token, r, b, n, page) for b, n in enumerate(lengths)] for r in range(R)]


def test_blocks_that_share_a_cache_are_alike(dev):
    one = PagedAttentionBlock(128, 2, 1, rows=2, seqs=2, pages=4, cols=2, device=dev)
    with pytest.raises(ValueError):
        PagedAttentionBlock(128, 2, 1, rows=2, seqs=2, pages=5, cols=2, device=dev, like=one)
    with pytest.raises(ValueError):
        PagedAttentionBlock(128, 2, 1, rows=3, seqs=2, pages=4, cols=2, R=2, device=dev)
    with pytest.raises(ValueError):
        PagedAttentionBlock(128, 2, 1, rows=2, seqs=3, pages=4, cols=2, device=dev)


def busy(dev, stream):
    """Work of some tens of milliseconds on the stream: what is not ordered behind it runs first."""
    with torch.cuda.stream(stream):
        a = torch.ones(8192, 8192, dtype=BF, device=dev)
        for _ in range(30):
            a @ a


def bits(x):
    return x.contiguous().view(torch.uint8)


def problem(dev, kept, lengths, new, seed=0, hq=16, hk=2, D=128, R=2, page=32, window=0, sinks=0):
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache=kept, window=window, sinks=sinks)
    cache = Cache(dev, d, lengths, new, seed)
    batch, rows = cache.batch(dev), sum(new)
    g = torch.Generator().manual_seed(seed + 1)
    q = [torch.randn(rows, hq * D, generator=g).to(BF).to(dev) for _ in range(R)]
    o = [torch.full((rows, hq * D), NAN, dtype=BF, device=dev) for _ in range(R)]
    ws = workspace(dev, d, batch, rows)

    def call(stream=None, o=o, ws=ws):
        B.fo_paged_attention(d, batch, rows, q, cache.kc, cache.vc, o, ws, cache.ks, cache.vs, None, stream)
    return cache, q, o, ws, call


FEW = ([700, 33, 0, 1500], [1, 1, 1, 1])
MANY = ([700, 33, 0, 1500], [300, 33, 1, 4])


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch", [FEW, MANY])
def test_work_is_on_the_calls_stream(dev, batch, kept):
    cache, q, o, ws, call = problem(dev, kept, *batch)
    call()
    want = [x.clone() for x in o]
    side = torch.cuda.Stream()
    right = [x.clone() for x in q]
    for x in q:
        x.zero_()
    torch.cuda.synchronize()
    busy(dev, side)
    with torch.cuda.stream(side):
        for x, y in zip(q, right):
            x.copy_(y)
    call(side)
    side.synchronize()
    assert B.fo_ops_status_query(ws, side)[0] == 0
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(o, want))


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
def test_two_graphs_with_workspaces_of_their_own_at_once(dev, kept):
    calls = [problem(dev, kept, *batch, seed=s) for s, batch in enumerate((FEW, MANY))]
    want, graphs, streams = [], [], [torch.cuda.Stream() for _ in calls]
    for _, _, o, _, call in calls:
        call()
        want.append([x.clone() for x in o])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(torch.cuda.current_stream())
        graphs.append(graph)
    for _, _, o, _, _ in calls:
        for x in o:
            x.fill_(NAN)
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, _, o, ws, _), w in zip(calls, want):
        assert B.fo_ops_status_query(ws)[0] == 0
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(o, w))


def test_one_workspace_serves_calls_of_all_kinds_in_turn(dev):
    """Calls that follow one another on a stream may share a workspace as large as the largest needs."""
    calls = [problem(dev, kept, *batch, seed=s, D=D) for s, (kept, batch, D) in enumerate(
        (("bf16", FEW, 128), ("bf16", MANY, 128), ("e4m3", MANY, 64), ("e4m3", FEW, 64), ("bf16", ([40], [40]), 64)))]
    ws = max((c[3] for c in calls), key=lambda w: w.numel())
    want = []
    for _, _, o, _, call in calls:
        call()
        want.append([x.clone() for x in o])
    for i in (0, 1, 2, 3, 4, 1, 0, 2, 0, 3, 4, 4, 1):
        for x in calls[i][2]:
            x.fill_(NAN)
        calls[i][4](ws=ws)
        assert B.fo_ops_status_query(ws)[0] == 0
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(calls[i][2], want[i])), i


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
def test_places_that_32_bits_do_not_count(dev, kept):
    """The sequences' pages are the cache's last, more than 2^32 values (bf16: 2^33 bytes) from its first."""
    for lengths, new in (([500, 33], [1, 1]), ([500, 33], [100, 33])):
        d = B.fo_paged_desc(8, 2, page=64, cache=kept)
        cache = Cache(dev, d, lengths, new, seed=2, big=(1 << 32) // (2 * 64 * 128) + 40)
        cache.table = torch.from_numpy(cache.table_all).to(dev)
        batch, rows = cache.batch(dev), sum(new)
        g = torch.Generator().manual_seed(3)
        draw = lambda n: [torch.randn(rows, n * 128, generator=g).to(BF).to(dev)]  # noqa: E731
        q, k, v, o = draw(8), draw(2), draw(2), [torch.empty(rows, 1024, dtype=BF, device=dev)]
        ws = workspace(dev, d, batch, rows)
        # the new tokens anew, of which the cache then holds what the oracle sees
        B.fo_kv_append(d, None, batch, rows, q, k, v, q, cache.kc, cache.vc, cache.ks, cache.vs, None, ws)
        B.fo_paged_attention(d, batch, rows, q, cache.kc, cache.vc, o, ws, cache.ks, cache.vs)
        assert B.fo_ops_status_query(ws)[0] == 0
        at = 0
        for b, (n, m) in enumerate(zip(lengths, new)):
            for x, c, s, keep in ((k, cache.kc, cache.ks, cache.k), (v, cache.vc, cache.vs, cache.v)):
                mine = x[0][at:at + m].view(m, 2, 128)
                if kept == "e4m3":
                    scale = (mine.float().abs().amax(dim=2) * np.float32(1 / 448)).clamp(min=2.0 ** -126)
                    mine = (mine.float() / scale[..., None]).to(E4M3).double() * scale[..., None].double()
                keep[0][b][n - m:] = f64(mine)
            at += m
        held_to_the_oracle(cache, [f64(q[0])], [f64(o[0])], None)
        del cache


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
def test_sequences_that_share_pages(dev, kept, new):
    """Sequences with the same beginning, kept once, and the same sequence twice."""
    cache, q, o, ws, call = problem(dev, kept, [200], [new], hq=8, R=1)
    call()
    table = torch.cat([cache.table] * 3)
    lengths, rows = [200, 200, 160], 3 * new
    q3 = [torch.cat([q[0]] * 3)]
    table[2] = torch.from_numpy(cache.table_all[0]).to(dev)
    batch = B.fo_paged_batch(whole(lengths, dev), table, cache.pages, starts=whole(first_rows([new] * 3), dev), max_new=new)
    o3, ws = [torch.empty(rows, 1024, dtype=BF, device=dev)], workspace(dev, cache.d, batch, rows)
    B.fo_paged_attention(cache.d, batch, rows, q3, cache.kc, cache.vc, o3, ws, cache.ks, cache.vs)
    assert B.fo_ops_status_query(ws)[0] == 0
    short = type("", (), dict(d=cache.d, lengths=[200, 200, 160], new=[new] * 3, k=[[cache.k[0][0], cache.k[0][0], cache.k[0][0][:160]]],
                              v=[[cache.v[0][0], cache.v[0][0], cache.v[0][0][:160]]]))
    held_to_the_oracle(short, [f64(q3[0])], [f64(o3[0])], None)


LONG = [  # R, heads_q, heads_k, D, kept, lengths, new, window: pairs cut into many parts
    (1, 8, 1, 128, "bf16", [20000], [5], 0),
    (1, 32, 1, 128, "e4m3", [9000, 300, 1], [4, 200, 1], 0),
    (2, 8, 2, 64, "e4m3", [6000, 40], [300, 40], 0),
    (1, 8, 1, 64, "bf16", [12000], [3], 7000),
    (1, 2, 1, 128, "bf16", [5000, 5000], [130, 9], 0),
]


@pytest.mark.parametrize("case", LONG)
def test_prompts_that_are_cut(dev, case):
    R, hq, hk, D, kept, lengths, new, window = case
    cache, q, o, ws, call = problem(dev, kept, lengths, new, seed=7, hq=hq, hk=hk, D=D, R=R, page=128, window=window, sinks=5 if window else 0)
    call()
    assert B.fo_ops_status_query(ws) == (0, [0, 0, 0, 0])
    held_to_the_oracle(cache, [f64(x) for x in q], [f64(x) for x in o], None)


def test_what_is_wrong_in_a_prompt_is_reported_and_harms_no_other(dev):
    d = B.fo_paged_desc(16, 2, page=16)
    lengths, new = [300, 200, 60], [40, 150, 20]
    for what, starts, change in ((1, None, (1, 3, 99)), (1, None, (1, 6, -1)), (2, None, None), (3, [0, 300, 190, 210], None),
                                 (3, [0, -1, 190, 210], None), (3, [0, 210, 0, 210], None), (4, None, None)):
        cache = Cache(dev, d, lengths, new, seed=9)
        rows = 210
        if change:
            cache.table[change[0], change[1]] = change[2]
        held = whole(lengths if what != 4 else [300, 4000, 60], dev)
        batch = B.fo_paged_batch(held, cache.table, cache.pages, starts=whole(starts or first_rows(new), dev), max_new=149 if what == 2 else 150)
        g = torch.Generator().manual_seed(4)
        q = [torch.randn(rows, 2048, generator=g).to(BF).to(dev)]
        o = [torch.zeros(rows, 2048, dtype=BF, device=dev)]
        ws = workspace(dev, d, batch, rows)
        B.fo_paged_attention(d, batch, rows, q, cache.kc, cache.vc, o, ws)
        code, info = B.fo_ops_status_query(ws)
        assert code == B.FO_ERR_SHAPE and info[2] == what and (info[1] == 1 or what == 3), (what, info)
        if what != 3:
            one = Cache(dev, d, lengths, new, seed=9)
            for b, lo in ((0, 0), (2, 190)):
                at = type("", (), dict(d=d, lengths=[lengths[b]], new=[new[b]], k=[[one.k[0][b]]], v=[[one.v[0][b]]]))
                held_to_the_oracle(at, [f64(q[0])[lo:]], [f64(o[0])[lo:]], None)
        # the workspace is as good as new
        again = Cache(dev, d, lengths, new, seed=9)
        good = again.batch(dev)
        B.fo_paged_attention(d, good, rows, q, again.kc, again.vc, o, ws)
        assert B.fo_ops_status_query(ws)[0] == 0
        held_to_the_oracle(again, [f64(q[0])], [f64(o[0])], None)


def test_calls_without_the_native_marshalling_are_the_same(dev, monkeypatch):
    for kept in ("bf16", "e4m3"):
        cache, q, o, ws, call = problem(dev, kept, *FEW)
        call()
        want = [x.clone() for x in o]

        class Plain:
            def __getattr__(self, name):
                return lambda *a: -1
        monkeypatch.setattr(B, "_marshal", Plain())
        call()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(o, want))
        d, rows = cache.d, len(q[0])
        full = torch.from_numpy(cache.table_all).to(dev)
        batch = B.fo_paged_batch(whole(cache.lengths, dev), full, cache.pages)
        k = [x[:, :256].contiguous() for x in q]
        got = []
        for marshal in (Plain(), None):
            monkeypatch.setattr(B, "_marshal", marshal)
            copy = lambda xs: None if xs is None else [x.clone() for x in xs]  # noqa: E731
            kc, vc, ks, vs, out = copy(cache.kc), copy(cache.vc), copy(cache.ks), copy(cache.vs), copy(q)
            B.fo_kv_append(d, None, batch, rows, q, k, k, out, kc, vc, ks, vs, None, ws)
            got.append(kc + vc + (ks or []) + (vs or []) + out)
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(*got))
        monkeypatch.undo()


MANY_SEQUENCES = [  # seqs, new, longest, heads_q, heads_k, D, page: more than a block of the plan has threads, and pairs than that
    (400, 1, 150, 4, 2, 64, 16),
    (1800, 3, 60, 8, 1, 64, 16),
    (1024, 5, 40, 4, 1, 128, 32),
    (1100, 1, 90, 2, 2, 128, 16),
]


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", MANY_SEQUENCES)
def test_many_sequences(dev, case, kept):
    seqs, most, longest, hq, hk, D, page = case
    g = np.random.default_rng(seqs)
    lengths = [int(n) for n in g.integers(0, longest + 1, seqs)]
    new = [int(m) for m in g.integers(0, most + 1, seqs)] if most > 1 else [1] * seqs
    new = [min(m, n) if most > 1 else m for m, n in zip(new, lengths)]
    new[-1] = max(new[-1], 1)
    cache, q, o, ws, call = problem(dev, kept, lengths, new, seed=5, hq=hq, hk=hk, D=D, R=1, page=page)
    call()
    assert B.fo_ops_status_query(ws) == (0, [0, 0, 0, 0])
    held_to_the_oracle(cache, [f64(x) for x in q], [f64(x) for x in o], None)


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1), (0, 2 ** 31 - 1), (1, 1)])
@pytest.mark.parametrize("new", [[1, 1], [90, 33]])
def test_the_largest_windows_and_sinks(dev, kept, window, sinks, new):
    cache, q, o, ws, call = problem(dev, kept, [200, 33], new, hq=4, hk=2, D=64, R=1, window=window, sinks=sinks)
    call()
    assert B.fo_ops_status_query(ws)[0] == 0
    held_to_the_oracle(cache, [f64(x) for x in q], [f64(x) for x in o], None)


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
def test_sixteen_ranks_prompts(dev, kept):
    cache, q, o, ws, call = problem(dev, kept, [150, 0, 20], [40, 0, 20], hq=3, hk=1, D=64, R=16)
    call()
    assert B.fo_ops_status_query(ws)[0] == 0
    held_to_the_oracle(cache, [f64(x) for x in q], [f64(x) for x in o], None)


def test_a_batch_in_which_nothing_is_new_touches_nothing(dev):
    d = B.fo_paged_desc(32, 2, page=16)
    cache = Cache(dev, d, [40, 0, 7], [1, 0, 1])
    for starts, lengths in (([0, 0, 0, 0], [40, 0, 7]), ([0, 0, 0, 0], [0, 0, 0]), ([3, 3, 3, 3], [0, 5, 0])):
        batch = B.fo_paged_batch(whole(lengths, dev), cache.table, cache.pages, starts=whole(starts, dev), max_new=8)
        o = [torch.full((6, 32 * 128), NAN, dtype=BF, device=dev)]
        ws = workspace(dev, d, batch, 6)
        B.fo_paged_attention(d, batch, 6, [torch.ones_like(o[0])], cache.kc, cache.vc, o, ws)
        assert B.fo_ops_status_query(ws)[0] == 0 and torch.isnan(o[0].float()).all()
        kept = [x.clone() for x in cache.kc + cache.vc]
        part = [torch.ones(6, 256, dtype=BF, device=dev)]
        B.fo_kv_append(d, None, batch, 6, [torch.ones_like(o[0])], part, part, o, cache.kc, cache.vc, ws=ws)
        assert B.fo_ops_status_query(ws)[0] == 0 and torch.isnan(o[0].float()).all()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(kept, cache.kc + cache.vc))


@pytest.mark.parametrize("spread", [4, 20, 30])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_values_of_all_magnitudes_in_8_bits(dev, spread, new):
    """Scales of tokens 2^spread above and below one: weights times scales, and values in the prompts' kernel, are f16, each
    off by 2^-11 of it, or, below 2^-14 with the largest magnitude at 2^8 (values) and 2^15 (weights times scales), by
    2^-25: 2^-31 of the largest value at most, both together."""
    hq, D, n = 8, 128, 300
    cache, q, o, ws, call = problem(dev, "e4m3", [n], [new], seed=1, hq=hq, hk=1, D=D, R=1, page=16)
    g = torch.Generator().manual_seed(2)
    mult = torch.exp2(torch.randint(-spread, spread + 1, (n,), generator=g).float())
    pg, slot = P.places(cache.table_all[0], n, 16)
    pg, slot = torch.from_numpy(pg.astype(np.int64)).to(dev), torch.from_numpy(slot).to(dev)
    cache.vs[0][pg, :, slot] *= mult.to(dev)[:, None]
    values = cache.v[0][0] * mult.double().numpy()[:, None, None]
    call()
    want, _, size, far = P.attention(f64(q[0]).reshape(new, hq, D), cache.k[0][0], values, new, 0, 0)
    score = (D + 8) * U * far + 2.0 ** -22
    bound = (2.0 ** -10 + 2 * score[..., None] + (2 * n + 8) * U) * size + 2.0 ** -31 * np.abs(values).max() + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)
    assert np.all(np.abs(f64(o[0]).reshape(want.shape) - want) <= bound)


@pytest.mark.parametrize("batch", [FEW, MANY])
def test_a_workspace_that_is_too_small_is_refused(dev, batch):
    cache, q, o, ws, call = problem(dev, "bf16", *batch)
    with pytest.raises(ValueError, match="smaller"):
        call(ws=ws[:-1])
    call()
    assert B.fo_ops_status_query(ws)[0] == 0
