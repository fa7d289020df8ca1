"""Appending to a paged cache, and attention over it, against the fp64 oracle.

Tolerances. Append: the rotation as in the rotary positions' own tests (cos and sin off by 8 u, u = 2^-24, and by the
frequency's rounding times the position), then half a step of bf16, 2^-8, or of e4m3, 2^-4 of a normal value and 2^-10 of
the smallest normal one below it.
Attention: a score is a sum of D products in fp32, off by at most (D + 8) u of the sum of their magnitudes (`far`, scaled;
the 8 for the scale, the change to base 2 and the difference from the maximum), and 2^x by 2^-22 of itself; both change a
weight and the weights' sum, so a result by twice that of `size` (the weights' sum over |v|). Sums over n keys add n u to
each of numerator and denominator. A weight is rounded to bf16 (2^-8 of it, so 2^-8 of `size`), the result once (2^-8 of it).
A column's 8-bit scale adds one more rounding of fp32. With more than 16 rows for a key head, an 8-bit cache's values times
their scales over a power of two become f16, and so do weights: two roundings of 2^-11 in place of the
one of 2^-8. lse: the scores' and the sum's errors, and 4 u of itself.
"""
import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from oracle import layer_ops as O
from oracle import paged as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn
NAN = float("nan")


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


def whole(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def first_rows(new):
    return [0] + np.cumsum(new).tolist()


class Cache:
    """R ranks' caches whose every place is NaN but those that a new token of `lengths`, `new` sees, which hold random
    values (self.k, self.v [r][b]: what they stand for); entries of the table that nobody needs name no page."""

    def __init__(self, dev, d, lengths, new, seed=0, spare=2, big=None):
        g = torch.Generator().manual_seed(seed)
        self.d, self.lengths, self.new, page = d, lengths, new, d.page
        cols = max(1, max([-(-max(n, 0) // page) for n in lengths], default=1)) + 1
        need = sum(-(-max(n, 0) // page) for n in lengths)
        self.pages = big or need + spare
        order = torch.randperm(self.pages, generator=g)[:need].tolist() if not big else list(range(self.pages - need, self.pages))
        table, at = np.full((len(lengths), cols), -7, dtype=np.int32), 0
        self.table_all = table.copy()
        self.k, self.v = ([[] for _ in range(d.R)] for _ in range(2))
        eight = d.cache_dtype == 1
        shape = (self.pages, d.heads_k, page, d.head_dim)
        fresh = (lambda: torch.full(shape, 0x7F, dtype=torch.uint8, device=dev).view(E4M3)) if eight else \
            (lambda: torch.full(shape, NAN, dtype=BF, device=dev))
        self.kc, self.vc = ([fresh() for _ in range(d.R)] for _ in range(2))
        scales = lambda: [torch.full(shape[:3], NAN, device=dev) for _ in range(d.R)] if eight else None  # noqa: E731
        self.ks, self.vs = scales(), scales()
        for b, (n, m) in enumerate(zip(lengths, new)):
            held = -(-max(n, 0) // page)
            self.table_all[b, :held] = order[at:at + held]
            at += held
            m = min(m, max(n, 0))
            seen = P.sees(n, m, d.window, d.sinks).any(axis=0) if m else np.zeros(max(n, 0), dtype=bool)
            for p in range(held):
                if seen[p * page:(p + 1) * page].any():
                    table[b, p] = self.table_all[b, p]
            pg, slot = P.places(self.table_all[b], max(n, 0), page)
            pg, slot = torch.from_numpy(pg[seen].astype(np.int64)).to(dev), torch.from_numpy(slot[seen]).to(dev)
            for r in range(d.R):
                for c, s, keep in ((self.kc, self.ks, self.k), (self.vc, self.vs, self.v)):
                    x = torch.randn(int(seen.sum()), d.heads_k, d.head_dim, generator=g) * torch.exp(0.3 * torch.randn(1, 1, d.head_dim, generator=g))
                    if eight:
                        scale = (x.abs().amax(dim=2) / 448.0).clamp(min=2.0 ** -126)
                        q = (x / scale[..., None]).to(E4M3)
                        c[r].view(torch.uint8)[pg, :, slot] = q.view(torch.uint8).to(dev)
                        s[r][pg, :, slot] = scale.to(dev)
                        x = q.double() * scale[..., None].double()
                    else:
                        x = x.to(BF)
                        c[r][pg, :, slot] = x.to(dev)
                    full = np.zeros((max(n, 0), d.heads_k, d.head_dim))
                    full[seen] = x.double().numpy()
                    keep[r].append(full)
        self.table = torch.from_numpy(table).to(dev)

    def batch(self, dev, starts=True):
        many = starts and (max(self.new, default=1) > 1 or min(self.new, default=1) < 1 or starts == "always")
        return B.fo_paged_batch(whole(self.lengths, dev), self.table, self.pages,
                                starts=whole(first_rows(self.new), dev) if many else None, max_new=max([1] + self.new) if many else 1)


def workspace(dev, d, batch, rows):
    ws = torch.empty(B.fo_paged_attention_workspace(d, batch.seqs, rows, batch.max_new), dtype=torch.uint8, device=dev)
    B.fo_ops_workspace_init(ws)
    return ws


def held_to_the_oracle(cache, q, o, lse, first=0):
    """Every row of every sequence against the oracle (q, o, lse: lists of fp64 [rows, heads * D], [rows, heads])."""
    d, at = cache.d, first
    for b, (n, m) in enumerate(zip(cache.lengths, cache.new)):
        for r in range(d.R):
            gone = max(0, m - max(n, 0))                     # rows before the sequence's beginning
            rows = slice(at + gone, at + m)
            assert np.all(o[r][at:at + gone] == 0) and (lse is None or np.all(lse[r][at:at + gone] == -np.inf))
            if m == gone:
                continue
            want, wl, size, far = P.attention(q[r][rows].reshape(m - gone, d.heads_q, d.head_dim), cache.k[r][b], cache.v[r][b], m - gone,
                                              d.window, d.sinks, d.scale or None)
            got = o[r][rows].reshape(want.shape)
            score = (d.head_dim + 8) * U * far + 2.0 ** -22
            bound = (2.0 ** -8 + 2 * score[..., None] + (2 * n + 8) * U) * size + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)
            assert np.all(np.abs(got - want) <= bound), (b, r, np.max(np.abs(got - want) / np.maximum(bound, 1e-300)))
            if lse is not None:
                off = score + (n + 8) * U + 4 * U * np.abs(wl)
                assert np.all(np.abs(lse[r][rows] - wl) <= off), (b, r)
        at += m


def attend(dev, d, lengths, new, seed=0, starts=True, wide=0, with_lse=True, tail=2):
    cache = Cache(dev, d, lengths, new, seed)
    batch, rows = cache.batch(dev, starts), sum(new) + tail
    g = torch.Generator().manual_seed(seed + 1)
    width = d.heads_q * d.head_dim
    whole_q = [torch.randn(rows, width + wide, generator=g).to(BF).to(dev) for _ in range(d.R)]
    whole_o = [torch.full((rows, width + wide), NAN, dtype=BF, device=dev) for _ in range(d.R)]
    q, o = [x[:, wide:] for x in whole_q], [x[:, wide:] for x in whole_o]
    lse = [torch.full((rows, d.heads_q), NAN, device=dev) for _ in range(d.R)] if with_lse else None
    ws = workspace(dev, d, batch, rows)
    call = lambda: B.fo_paged_attention(d, batch, rows, q, cache.kc, cache.vc, o, ws, cache.ks, cache.vs, lse)  # noqa: E731
    call()
    assert B.fo_ops_status_query(ws) == (0, [0, 0, 0, 0])
    held_to_the_oracle(cache, [f64(x) for x in q], [f64(x) for x in o], [f64(x) for x in lse] if lse else None)
    for x in whole_o:                                        # rows behind the last sequence, and what lies beside o
        assert torch.isnan(x[sum(new):].float()).all() and torch.isnan(x[:, :wide].float()).all()
    if lse:
        assert all(torch.isnan(x[sum(new):]).all() for x in lse)
    before = [x.clone() for x in o]
    call()
    assert all(torch.equal(x[:sum(new)].view(torch.int16), y[:sum(new)].view(torch.int16)) for x, y in zip(o, before))
    return cache


DECODE = [  # R, heads_q, heads_k, D, page, lengths, new
    (1, 1, 1, 64, 16, [1], [1]),
    (1, 4, 4, 128, 16, [1, 2, 0, 15, 16, 17], [1] * 6),
    (2, 8, 2, 128, 64, [63, 64, 65, 129], [1] * 4),
    (1, 32, 8, 128, 64, [512, 31, 33, 257, 0, 1000], [1] * 6),
    (1, 16, 1, 64, 32, [700], [1]),
    (3, 7, 1, 128, 256, [255, 256, 257], [1] * 3),
    (1, 64, 1, 128, 128, [300, 5], [1] * 2),
    (1, 5, 5, 64, 16, [3000, 1], [1] * 2),
    (1, 20, 4, 128, 32, [100, 99, 3, 40], [4, 1, 3, 2]),
    (2, 16, 2, 128, 16, [300, 5, 64, 70], [7, 5, 6, 0]),
    (1, 24, 8, 64, 64, [128, 2, 0], [5, 3, 2]),           # more new tokens than tokens: rows that see nothing
    (16, 2, 1, 64, 16, [40, 9], [1] * 2),
    (1, 32, 2, 128, 16, [200, 100], [2, 1]),
    (1, 16, 1, 128, 64, [900, 77], [4, 4]),
]
SIGHTS = [(0, 0), (1, 0), (16, 4), (100, 0), (64, 130), (33, 1), (5000, 3)]


@pytest.mark.parametrize("window,sinks", SIGHTS)
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", DECODE)
def test_few_new_tokens(dev, case, kept, window, sinks):
    R, hq, hk, D, page, lengths, new = case
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache=kept, window=window, sinks=sinks)
    attend(dev, d, lengths, new, seed=hq + D)


PROMPTS = [
    (1, 1, 1, 128, 16, [17], [17]),
    (1, 2, 1, 64, 16, [130, 1, 0, 200], [130, 1, 0, 70]),
    (1, 4, 2, 128, 64, [300, 128, 500], [300, 128, 129]),
    (2, 3, 1, 128, 32, [257, 90], [200, 90]),
    (1, 7, 1, 64, 128, [150], [149]),
    (1, 8, 1, 128, 256, [400, 600], [100, 33]),
    (1, 64, 1, 128, 16, [80, 7], [5, 7]),
    (1, 20, 4, 64, 16, [100, 30], [64, 40]),              # rows before the beginning of the second
    (1, 2, 1, 128, 32, [2500, 130, 5], [70, 65, 1]),      # one long context: its steps are cut and joined
    (2, 20, 1, 64, 16, [1800], [33]),
]


@pytest.mark.parametrize("window,sinks", SIGHTS)
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", PROMPTS)
def test_prompts(dev, case, kept, window, sinks):
    R, hq, hk, D, page, lengths, new = case
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache=kept, window=window, sinks=sinks)
    attend(dev, d, lengths, new, seed=hq + D + 1)


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 1, 2], [90, 100, 1]])
def test_rows_that_are_parts_of_wider_ones_and_a_scale_of_the_callers(dev, new):
    d = B.fo_paged_desc(8, 2, head_dim=64, page=32, scale=0.3)
    attend(dev, d, [90, 200, 33], new, wide=72, with_lse=False, tail=0)
    attend(dev, d, [90, 200, 33], new, starts="always", with_lse=False)


# ------------------------------------------------------------------ append

def turned(x, pos, d, rope):
    """The oracle's rotation of x [rows, heads * D] and how far a correct one may be off before it is stored."""
    if rope is None:
        return x, np.zeros_like(x)
    f, factor = O.rope_frequencies(rope.rot_dim, rope.base)
    layout = "half" if rope.layout == 0 else "interleaved"
    want = O.rope(x, pos, f, factor, d.head_dim, layout)
    v = np.abs(x.reshape(len(x), -1, d.head_dim))
    size, pairs = np.zeros_like(v), len(f)
    ia = np.arange(pairs) if layout == "half" else 2 * np.arange(pairs)
    ib = ia + pairs if layout == "half" else ia + 1
    size[:, :, ia] = size[:, :, ib] = v[:, :, ia] + v[:, :, ib]
    far = 8 * U + 16 * 2.0 ** -53 * (np.max(np.abs(pos)) if len(pos) else 0)
    return want, far * size.reshape(x.shape)


APPEND = [  # R, heads_q, heads_k, D, page, rot, layout, lengths, new, wide
    (1, 1, 1, 64, 16, 64, "half", [1], [1], 0),
    (2, 8, 2, 128, 64, 128, "half", [63, 64, 65, 0, 4], [1] * 5, 0),
    (1, 32, 8, 128, 16, 64, "interleaved", [100, 3, 40, 0, 16], [37, 3, 0, 2, 16], 0),
    (1, 4, 4, 128, 32, 128, "interleaved", [33, 200], [33, 7], 4),
    (3, 6, 2, 64, 256, 32, "half", [300, 9], [290, 9], 0),
    (1, 5, 1, 64, 128, 20, "half", [50, 20], [20, 30], 2),         # a token before the beginning
    (1, 3, 3, 128, 16, 6, "half", [17, 5], [5, 5], 1),             # odd strides, three pairs
    (2, 2, 1, 64, 16, 10, "interleaved", [17, 5], [5, 5], 3),
    (1, 64, 1, 128, 64, None, "half", [70], [70], 0),              # nothing turned
    (16, 1, 1, 128, 16, 128, "half", [5, 6], [1, 1], 0),
]


@pytest.mark.parametrize("given", [None, torch.int32, torch.int64])
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", APPEND)
def test_append(dev, case, kept, given):
    R, hq, hk, D, page, rot, layout, lengths, new, wide = case
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache=kept)
    rope = None if rot is None else B.fo_rope_desc(D, hq, hk, hk, R=R, rot_dim=rot, layout=layout, base=500000.0)
    cache = Cache(dev, d, lengths, [0] * len(lengths), seed=3)
    cache.table, cache.new = torch.from_numpy(cache.table_all).to(dev), new
    batch, rows = cache.batch(dev), sum(new) + 1
    g = torch.Generator().manual_seed(5)
    heads = (hq, hk, hk)
    packed = [torch.randn(rows, sum(heads) * D + wide, generator=g).to(BF).to(dev) for _ in range(R)]
    parts = [[p[:, :sum(heads) * D].split([n * D for n in heads], dim=1)[j] for p in packed] for j in range(3)]
    q_out = [torch.full((rows, hq * D), NAN, dtype=BF, device=dev) for _ in range(R)]
    where = [(b, n - m + i) for b, (n, m) in enumerate(zip([max(n, 0) for n in lengths], new)) for i in range(m)]
    pos = np.array([p for _, p in where], dtype=np.float64)
    at = None
    if given is not None:
        at = torch.randint(-5, 1 << 20, (rows,), generator=g, dtype=given)
        pos, at = at.numpy().astype(np.float64)[:len(where)], at.to(dev)
    ws = workspace(dev, d, batch, rows)
    B.fo_kv_append(d, rope, batch, rows, *parts, q_out, cache.kc, cache.vc, cache.ks, cache.vs, at, ws)
    assert B.fo_ops_status_query(ws) == (0, [0, 0, 0, 0])
    kept_at = [(i, cache.table_all[b, p // page], p % page) for i, (b, p) in enumerate(where) if p >= 0]
    taken = np.zeros((cache.pages, page), dtype=bool)
    for _, pg, slot in kept_at:
        taken[pg, slot] = True
    for r in range(R):
        used = len(where)
        want, off = turned(f64(parts[0][r])[:used], pos, d, rope)
        assert np.all(np.abs(f64(q_out[r])[:used] - want) <= off + 2.0 ** -8 * (np.abs(want) + off))
        assert torch.isnan(q_out[r][used:].float()).all()
        for j, c, s in ((1, cache.kc, cache.ks), (2, cache.vc, cache.vs)):
            x = f64(parts[j][r])[:used]
            want, off = turned(x, pos, d, rope) if j == 1 else (x, np.zeros_like(x))
            want, off = (v.reshape(used, hk, D) for v in (want, off))
            got, i = f64(c[r].float()), [i for i, _, _ in kept_at]
            mine = np.array([got[pg, :, slot] for _, pg, slot in kept_at]).reshape(len(i), hk, D)
            if kept == "bf16":
                assert np.all(np.abs(mine - want[i]) <= off[i] + 2.0 ** -8 * (np.abs(want[i]) + off[i]) * (j == 1))
            else:
                quotient, scale = P.in_8_bits(want[i])
                sc = f64(s[r])
                held = np.array([sc[pg, :, slot] for _, pg, slot in kept_at]).reshape(len(i), hk)
                # The scale is off by its largest value's error and two roundings; the quotient by both's.
                rel = off[i].max(axis=2) / np.maximum(np.abs(want[i]).max(axis=2), 1e-300) + 4 * U
                assert np.all(np.abs(held - scale) <= rel * scale)
                moved = off[i] / scale[..., None] + np.abs(quotient) * (rel[..., None] + 4 * U)
                assert np.all(np.abs(mine - quotient) <= moved + np.maximum(2.0 ** -4 * (np.abs(quotient) + moved), 2.0 ** -10))
                if j == 2:      # V is not turned: the very numbers of the formula in fp32
                    f = torch.from_numpy(x[i].reshape(len(i), hk, D)).float()
                    assert np.array_equal(held.astype(np.float32), (f.abs().amax(dim=2) * np.float32(1 / 448)).clamp(min=2.0 ** -126).numpy())
                assert np.isnan(np.moveaxis(sc, 1, 2)[~taken]).all()
            assert np.isnan(np.moveaxis(got, 1, 2)[~taken]).all()
    # In place, and what is turned beforehand by the rotary call alone, give the same bits.
    again = [p.clone() for p in packed]
    mine = [[p[:, :sum(heads) * D].split([n * D for n in heads], dim=1)[j] for p in again] for j in range(3)]
    keep = [x.clone() for x in cache.kc]
    B.fo_kv_append(d, rope, batch, rows, *mine, mine[0], cache.kc, cache.vc, cache.ks, cache.vs, at)
    bits = lambda x: x.contiguous().view(torch.uint8)  # noqa: E731
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(cache.kc, keep))
    assert all(torch.equal(bits(a[:used]), bits(b[:used])) for a, b in zip(mine[0], q_out))
    assert all(torch.equal(a[used:], b[used:]) and torch.equal(a[:, hq * D:], b[:, hq * D:]) for a, b in zip(again, packed))


def test_append_holds_nan_infinity_and_zeros_as_the_quantiser_does(dev):
    d = B.fo_paged_desc(1, 1, page=16, cache="e4m3")
    cache = Cache(dev, d, [4], [0])
    cache.table, cache.new = torch.from_numpy(cache.table_all).to(dev), [4]
    x = torch.randn(4, 128).to(BF)
    x[0] = 0
    x[1, 5] = NAN
    x[2, 7] = float("inf")
    x[3] = 2.0 ** -130
    x = x.to(dev)
    q, scale = torch.empty(4, 128, dtype=E4M3, device=dev), torch.empty(4, 1, device=dev)
    B.fo_quant_fp8(4, 128, [x], [q], [scale])
    B.fo_kv_append(d, None, cache.batch(dev), 4, [x], [x], [x], [x.clone()], cache.kc, cache.vc, cache.ks, cache.vs)
    page = int(cache.table_all[0, 0])
    for c, s in ((cache.kc, cache.ks), (cache.vc, cache.vs)):
        assert torch.equal(c[0][page, 0, :4].view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(s[0][page, 0, :4].view(torch.int32), scale[:, 0].view(torch.int32))


# ------------------------------------------------------------------ what the device finds wrong

def test_what_is_wrong_on_the_device_is_reported_and_harms_no_other_sequence(dev):
    d = B.fo_paged_desc(4, 2, page=16, R=2)
    lengths, new = [40, 100, 60], [2, 3, 1]
    for what, starts, change, value in ((1, None, (1, 3, 99), 99), (1, None, (1, 6, -1), -1), (2, None, None, 3), (3, [0, 9, 5, 6], None, None),
                                        (3, [0, -1, 5, 6], None, None), (4, None, None, 4000)):
        cache = Cache(dev, d, lengths, new, seed=9)
        rows, first = 6, whole(starts or first_rows(new), dev)
        if change:
            cache.table[change[0], change[1]] = change[2]
        held = whole(lengths if what != 4 else [40, 4000, 60], dev)
        batch = B.fo_paged_batch(held, cache.table, cache.pages, starts=first, max_new=2 if what == 2 else 3)
        g = torch.Generator().manual_seed(4)
        q = [torch.randn(rows, 512, generator=g).to(BF).to(dev) for _ in range(2)]
        o = [torch.zeros(rows, 512, dtype=BF, device=dev) for _ in range(2)]
        ws = workspace(dev, d, batch, rows)
        B.fo_paged_attention(d, batch, rows, q, cache.kc, cache.vc, o, ws)
        code, info = B.fo_ops_status_query(ws)
        assert code == B.FO_ERR_SHAPE and info[2] == what and (info[3] == value or value is None), (what, info)
        assert info[1] == 1 or what == 3
        assert B.fo_ops_status_query(ws)[0] == 0
        if what != 3:
            for b, (lo, hi) in ((0, (0, 2)), (2, (5, 6))):
                one = Cache(dev, d, lengths, new, seed=9)
                one.lengths, one.new = [lengths[b]], [new[b]]
                one.k, one.v = [[x[b]] for x in one.k], [[x[b]] for x in one.v]
                held_to_the_oracle(one, [f64(x)[lo:hi] for x in q], [f64(x)[lo:hi] for x in o], None)
        if what == 1:
            B.fo_kv_append(d, None, B.fo_paged_batch(whole([40, 16 * change[1] + 3, 60], dev), cache.table, cache.pages, starts=first, max_new=3),
                           rows, q, [x[:, :256] for x in q], [x[:, :256] for x in q], o, cache.kc, cache.vc, ws=ws)
            assert B.fo_ops_status_query(ws) == (B.FO_ERR_SHAPE, [B.FO_ERR_SHAPE, 1, 1, value])
