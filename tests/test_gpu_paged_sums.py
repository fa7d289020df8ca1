"""What the attention over a paged cache carries from one tile of keys to the next: running maxima and sums, the powers of two
of an 8-bit cache's values, outputs that are rescaled; in single tiles, in items of many steps and in blocks with many
tiles, against the fp64 oracle.

Tolerances are the ones of the operator's own tests (test_gpu_paged.py), and of an 8-bit cache what its roundings leave:
weights become f16 (2^-11 of each), with more than 16 rows for a key head the values too, times their scale over a power of
two: the scale's share once and the product once (2^-11 each). Below f16's least normal number a weight, or a
value's scale, is off by 2^-25 of a range whose top is 2^15 (or 2^7) times a power of two not below the largest scale of the
values seen: with an e4m3 value of up to 448, 2^-31 of the largest value at most, for each value that the row sees. A
query's row becomes f16 with its largest magnitude in [128, 256): 2^-32 of that.
fp32 itself ends: a weight below 2^-126 is zero, and so is such a factor when tiles or parts are joined. Weights are at most
2^8 (the maximum moves late) and their sum is at least 1, so each of n values loses at most 2^8 * 2^-126 of the largest of
them: n 2^-118 max |v|. (Values that fall by 2^9 for each of 24 tiles whose weights grow as fast differ by 2^216: no fp32
weight reaches the first of them, whatever the order of the sums.)
"""
import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from oracle import paged as P
from test_gpu_paged import BF, E4M3, NAN, U, f64, first_rows, whole, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


class Kept:
    """R ranks' caches of keys(r, b) and values(r, b), [length, heads_k, D]; self.k, self.v: what they stand for in fp64."""

    def __init__(self, dev, d, lengths, keys, values, seed=0):
        self.d, self.lengths, page = d, lengths, d.page
        cols = max(-(-n // page) for n in lengths)
        need = sum(-(-n // page) for n in lengths)
        self.pages = need + 2
        order = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed))[:need].tolist()
        table = np.full((len(lengths), cols), -7, dtype=np.int32)
        for b, n in enumerate(lengths):
            held = -(-n // page)
            table[b, :held], order = order[:held], order[held:]
        eight = d.cache_dtype == 1
        shape = (self.pages, d.heads_k, page, d.head_dim)
        fresh = (lambda: torch.full(shape, 0x7F, dtype=torch.uint8, device=dev).view(E4M3)) if eight else \
            (lambda: torch.full(shape, NAN, dtype=BF, device=dev))
        self.kc, self.vc = ([fresh() for _ in range(d.R)] for _ in range(2))
        scales = lambda: [torch.full(shape[:3], NAN, device=dev) for _ in range(d.R)] if eight else None  # noqa: E731
        self.ks, self.vs = scales(), scales()
        self.k, self.v = ([[] for _ in range(d.R)] for _ in range(2))
        for b, n in enumerate(lengths):
            pg, slot = (torch.from_numpy(x.astype(np.int64)).to(dev) for x in P.places(table[b], n, page))
            for r in range(d.R):
                for c, s, held, x in ((self.kc, self.ks, self.k, keys(r, b)), (self.vc, self.vs, self.v, values(r, b))):
                    if eight:
                        scale = (x.abs().amax(dim=2) / 448.0).clamp(min=2.0 ** -126)
                        q = (x / scale[..., None]).to(E4M3)
                        c[r].view(torch.uint8)[pg, :, slot] = q.view(torch.uint8).to(dev)
                        s[r][pg, :, slot] = scale.to(dev)
                        x = q.double() * scale[..., None].double()
                    else:
                        x = x.to(BF)
                        c[r][pg, :, slot] = x.to(dev)
                    held[r].append(x.double().numpy())
        self.table = torch.from_numpy(table).to(dev)


def attend(dev, cache, new, q):
    """Results [r] of o [rows, heads * D] and lse [rows, heads]; two calls give the same bits."""
    d, rows = cache.d, sum(new)
    batch = B.fo_paged_batch(whole(cache.lengths, dev), cache.table, cache.pages, starts=whole(first_rows(new), dev), max_new=max(new))
    q = [x.to(dev) for x in q]
    o = [torch.full((rows, d.heads_q * d.head_dim), NAN, dtype=BF, device=dev) for _ in range(d.R)]
    lse = [torch.full((rows, d.heads_q), NAN, device=dev) for _ in range(d.R)]
    ws = workspace(dev, d, batch, rows)
    got = []
    for _ in range(2):
        B.fo_paged_attention(d, batch, rows, q, cache.kc, cache.vc, o, ws, cache.ks, cache.vs, lse)
        assert B.fo_ops_status_query(ws) == (0, [0, 0, 0, 0])
        got.append([x.clone() for x in o + lse])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got))
    return [f64(x) for x in o], [f64(x) for x in lse]


def held_to_the_oracle(cache, new, q, o, lse, rows_each=None, seed=0):
    """All rows against the oracle, or `rows_each` of each sequence, the first and the last among them."""
    d, at = cache.d, 0
    prompts = max(new) * (d.heads_q // d.heads_k) > 16
    g = np.random.default_rng(seed)
    for b, (n, m) in enumerate(zip(cache.lengths, new)):
        some = np.arange(m) if rows_each is None or rows_each >= m else \
            np.unique(np.concatenate([[0, m - 1], g.integers(0, m, rows_each - 2)]))
        seen = P.sees(n, m, d.window, d.sinks).any(axis=0)
        for r in range(d.R):
            k, v = cache.k[r][b], cache.v[r][b]
            group = d.heads_q // d.heads_k
            top = np.repeat(np.abs(v[seen]).max(axis=(0, 2)), group)[:, None]     # of a key head's values that are seen
            for i in some:
                p = n - m + i
                mine = f64(q[r][at + i]).reshape(1, d.heads_q, d.head_dim)
                want, wl, size, far = (x[0] for x in P.attention(mine, k[:p + 1], v[:p + 1], 1, d.window, d.sinks, d.scale or None))
                count = int(P.sees(p + 1, 1, d.window, d.sinks).sum())
                score, weights, least = (d.head_dim + 8) * U * far + 2.0 ** -22, 2.0 ** -8, 0.0
                if d.cache_dtype == 1:
                    key = np.repeat(np.abs(k[:p + 1]).sum(axis=2).max(axis=0), group)
                    score = score + 2.0 ** -32 * np.abs(mine[0]).max(axis=1) * key * (d.scale or d.head_dim ** -0.5)
                    weights, least = (3 if prompts else 1) * 2.0 ** -11 * (1 + 2.0 ** -9), count * 2.0 ** -31
                bound = (weights + 2 * score[:, None] + (2 * n + 8) * U) * size + (least + count * 2.0 ** -118) * top + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)
                got = o[r][at + i].reshape(want.shape)
                assert np.all(np.abs(got - want) <= bound), (b, r, i, np.max(np.abs(got - want) / np.maximum(bound, 1e-300)))
                off = score + (n + 8) * U + 4 * U * np.abs(wl)
                assert np.all(np.abs(lse[r][at + i] - wl) <= off), (b, r, i, np.max(np.abs(lse[r][at + i] - wl) / off))
        at += m


def draws(seed, hk, D, lengths):
    """A function of (rank, sequence) with standard normal keys or values [length, hk, D]."""
    def one(r, b):
        return torch.randn(lengths[b], hk, D, generator=torch.Generator().manual_seed(seed * 1000 + r * 100 + b))
    return one


def queries(seed, d, rows):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(rows, d.heads_q * d.head_dim, generator=g).to(BF) for _ in range(d.R)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (200, 33)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_each_32_values_of_an_8_bit_cache_have_a_power_of_two_of_their_own(dev, D, page, window, sinks):
    """It is the step's own, and there when the step's weights are made, whatever the steps before had in its place."""
    lengths, new, hq, hk, R = [1500, 700, 90], [900, 64, 90], 8, 2, 2
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache="e4m3", window=window, sinks=sinks)
    normal = draws(3, hk, D, lengths)
    g = torch.Generator().manual_seed(4)
    powers = torch.randint(-8, 9, (max(lengths) // 32 + 1, R), generator=g).float()

    def values(r, b):
        return normal(r, b) * torch.exp2(powers[:, r].repeat_interleave(32)[:lengths[b]])[:, None, None]
    cache = Kept(dev, d, lengths, draws(5, hk, D, lengths), values)
    q = queries(6, d, sum(new))
    o, lse = attend(dev, cache, new, q)
    held_to_the_oracle(cache, new, q, o, lse, rows_each=60)


@pytest.mark.parametrize("power", [20, 24, 27, 31, 40, 100])
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_scores_of_any_magnitude_have_weights_that_are_numbers(dev, kept, new, power):
    """Queries 2^power times ordinary ones, some rows of them, beside ordinary rows."""
    hq, D, lengths = 8, 64, [900, 70]
    d = B.fo_paged_desc(hq, 1, head_dim=D, page=16, cache=kept)
    cache = Kept(dev, d, lengths, draws(1, 1, D, lengths), draws(2, 1, D, lengths))
    q = queries(3, d, 2 * new)
    for x in q:
        x[::2] *= 2.0 ** power
    o, lse = attend(dev, cache, [new, new], q)
    held_to_the_oracle(cache, [new, new], q, o, lse)


@pytest.mark.parametrize("power", [10, 20, 30, 40, 60])
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_of_large_scores_without_roundings_the_largest_takes_all(dev, kept, new, power):
    """Queries and keys that are powers of two at one place each: scores are exact, and 2^power apart at least."""
    hq, D, n = 8, 64, 500
    d = B.fo_paged_desc(hq, 1, head_dim=D, page=16, cache=kept, scale=1.0)
    place = torch.randint(0, D, (n,), generator=torch.Generator().manual_seed(1))

    def keys(r, b):
        x = torch.zeros(n, 1, D)
        x[torch.arange(n), 0, place] = -448.0 * 2.0 ** (torch.arange(n) % 5 - 8)
        return x
    cache = Kept(dev, d, [n], keys, draws(2, 1, D, [n]))
    q = torch.zeros(new, hq, D)
    for i in range(new):
        for h in range(hq):
            q[i, h] = 2.0 ** power / 1.75
            q[i, h, place[(7 * i + 13 * h) % (n - new)]] = 0
    q = q.to(BF)
    o, lse = attend(dev, cache, [new], [q.view(new, -1)])
    for i in range(new):
        for h in range(hq):
            s = f64(q[i, h]) @ cache.k[0][0][:n - new + i + 1, 0].T
            top = np.flatnonzero(s == s.max())
            want = cache.v[0][0][top, 0].mean(axis=0)
            size = np.abs(cache.v[0][0][top, 0]).mean(axis=0)
            got = o[0][i].reshape(hq, D)[h]
            assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + (2 * n + 8) * U) * size + 2.0 ** -25)
            assert abs(lse[0][i, h] - s.max() - np.log(len(top))) <= (n + 8) * U + 4 * U * abs(s.max() + np.log(len(top)))


@pytest.mark.parametrize("scale", [1e-6, 4.0e-8, 1e-20, 1.2e-38, 1e-44])
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_scores_of_a_scale_near_zero_are_numbers(dev, kept, new, scale):
    """Queries that are zero, ordinary and large: a hidden key's weight is none, and the seen ones' are alike."""
    hq, D, lengths = 4, 128, [200, 70]
    d = B.fo_paged_desc(hq, 1, head_dim=D, page=16, cache=kept, scale=scale, window=50, sinks=3)
    cache = Kept(dev, d, lengths, draws(1, 1, D, lengths), draws(2, 1, D, lengths))
    q = queries(3, d, 2 * new)
    for x in q:
        x[0] = 0
        x[-1, :D] *= 2.0 ** -120
        x[-1, D:2 * D] *= 2.0 ** 60
        x[-1, 2 * D:3 * D] *= 2.0 ** -128
    o, lse = attend(dev, cache, [new, new], q)
    held_to_the_oracle(cache, [new, new], q, o, lse)


@pytest.mark.parametrize("spread", [6, 12, 20, 30])
@pytest.mark.parametrize("D", [64, 128])
def test_small_values_beside_hidden_large_ones_in_8_bits(dev, D, spread):
    """Prompts without a prefix: rows see few values, whose scales are 2^-spread to 2^spread of the ones they do not see."""
    lengths = [300, 33, 90]
    d = B.fo_paged_desc(8, 1, head_dim=D, page=32, cache="e4m3", window=60)
    normal = draws(1, 1, D, lengths)
    powers = torch.randint(-spread, spread + 1, (300,), generator=torch.Generator().manual_seed(3)).float()
    cache = Kept(dev, d, lengths, draws(2, 1, D, lengths), lambda r, b: normal(r, b) * torch.exp2(powers[:lengths[b]])[:, None, None])
    q = queries(4, d, sum(lengths))
    o, lse = attend(dev, cache, lengths, q)
    held_to_the_oracle(cache, lengths, q, o, lse)


@pytest.mark.parametrize("spread", [6, 12, 20, 30])
@pytest.mark.parametrize("D", [64, 128])
def test_small_values_beside_hidden_large_ones_among_few_tokens(dev, D, spread):
    lengths, new = [4, 3, 2, 70, 1], [4, 3, 2, 2, 1]
    d = B.fo_paged_desc(4, 1, head_dim=D, page=16, cache="e4m3", window=3)
    normal = draws(1, 1, D, lengths)
    powers = torch.randint(-spread, spread + 1, (70,), generator=torch.Generator().manual_seed(3)).float()
    cache = Kept(dev, d, lengths, draws(2, 1, D, lengths), lambda r, b: normal(r, b) * torch.exp2(powers[:lengths[b]])[:, None, None])
    q = queries(4, d, sum(new))
    o, lse = attend(dev, cache, new, q)
    held_to_the_oracle(cache, new, q, o, lse)


# ------------------------------------------------------------------ an 8-bit cache's own bound

def shapes():
    """The operator's own shapes, of sequences whose new tokens all are in the cache."""
    from test_gpu_paged import DECODE, PROMPTS
    for R, hq, hk, D, page, lengths, new in DECODE + PROMPTS:
        kept = [(n, m) for n, m in zip(lengths, new) if n >= m > 0]
        yield R, hq, hk, D, page, [n for n, _ in kept], [m for _, m in kept]


@pytest.mark.parametrize("window,sinks", [(0, 0), (16, 4), (64, 130), (33, 1)])
@pytest.mark.parametrize("case", list(shapes()))
def test_an_8_bit_cache_costs_what_its_roundings_cost(dev, case, window, sinks):
    R, hq, hk, D, page, lengths, new = case
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache="e4m3", window=window, sinks=sinks)
    cache = Kept(dev, d, lengths, draws(hq, hk, D, lengths), draws(hq + 1, hk, D, lengths))
    q = queries(2, d, sum(new))
    o, lse = attend(dev, cache, new, q)
    held_to_the_oracle(cache, new, q, o, lse, rows_each=40)


# ------------------------------------------------------------------ maxima that grow, outputs that are rescaled

def steps_of(by, each, lengths, hk, D, seed):
    """Keys whose first place alone counts: with queries of 4 there and a scale of 1/4 the score of token j is by * (j //
    each) / log2 e, plus what the other places, a tenth of normal ones, add."""
    def one(r, b):
        n = lengths[b]
        x = 0.1 * torch.randn(n, hk, D, generator=torch.Generator().manual_seed(seed + 10 * r + b))
        x[:, :, 0] = by / 1.4426950408889634 * (torch.arange(n) // each).float()[:, None]
        return x
    return one


def aligned_queries(seed, d, rows):
    q = queries(seed, d, rows)
    for x in q:
        x.view(rows, d.heads_q, d.head_dim)[:, :, 0] = 4
    return q


GROWTH = [  # lengths, new, heads_q, heads_k, R: blocks with several tiles, items with many steps
    ([6000, 4100, 5300, 4900] * 4, [1] * 16, 8, 4, 1),
    ([3000, 2100] * 3, [3] * 6, 10, 2, 2),
    ([1500, 700], [40, 700], 8, 2, 2),
    ([6000, 300], [1000, 300], 8, 2, 3),
]


@pytest.mark.parametrize("by", [9.0, 3.0, 7.9])
@pytest.mark.parametrize("kept,shrink", [("bf16", 0), ("bf16", 1), ("e4m3", 0)])
@pytest.mark.parametrize("case", GROWTH)
def test_scores_that_grow_from_tile_to_tile(dev, case, kept, shrink, by):
    """By 2^9 for each 128 keys (the maximum moves), 2^3 and just below 2^8 (it moves late); values that shrink as fast
    (`shrink`) leave the first tiles' share as large as the last's."""
    lengths, new, hq, hk, R = case
    D, each = 64, 128
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=32, cache=kept, scale=0.25)
    normal = draws(7, hk, D, lengths)

    def values(r, b):
        t = (torch.arange(lengths[b]) // each).float()
        return normal(r, b) * torch.exp2(-by * shrink * (t - t.max() / 2)).clamp(2.0 ** -100, 2.0 ** 100)[:, None, None]
    cache = Kept(dev, d, lengths, steps_of(by, each, lengths, hk, D, 3), values)
    q = aligned_queries(8, d, sum(new))
    o, lse = attend(dev, cache, new, q)
    held_to_the_oracle(cache, new, q, o, lse, rows_each=12)


@pytest.mark.parametrize("each,by", [(256, 9.0), (128, 8.0), (512, 20.0)])
@pytest.mark.parametrize("case", GROWTH)
def test_values_of_an_8_bit_cache_that_grow_from_tile_to_tile(dev, case, each, by):
    """By 2^by for each block of keys, whose scores fall as fast: all blocks' shares are alike, and the power of two that the
    weights are kept over moves with each."""
    lengths, new, hq, hk, R = case
    D = 64
    lengths = [min(n, int(110 / by) * each) for n in lengths]
    new = [min(m, n) for m, n in zip(new, lengths)]
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=32, cache="e4m3", scale=0.25)
    normal = draws(7, hk, D, lengths)

    def values(r, b):
        t = (torch.arange(lengths[b]) // each).float()
        return normal(r, b) * torch.exp2(by * (t - t.max() / 2)).clamp(2.0 ** -60, 2.0 ** 60)[:, None, None]
    cache = Kept(dev, d, lengths, steps_of(-by, each, lengths, hk, D, 3), values)
    q = aligned_queries(8, d, sum(new))
    o, lse = attend(dev, cache, new, q)
    held_to_the_oracle(cache, new, q, o, lse, rows_each=12)


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", GROWTH)
def test_peaked_rows(dev, case, kept):
    """Scores of a standard deviation of 12: most of a row's weight is one key's, wherever it lies."""
    lengths, new, hq, hk, R = case
    d = B.fo_paged_desc(hq, hk, head_dim=128, R=R, page=64, cache=kept)
    cache = Kept(dev, d, lengths, lambda r, b: 12 * draws(1, hk, 128, lengths)(r, b), draws(2, hk, 128, lengths))
    q = queries(3, d, sum(new))
    o, lse = attend(dev, cache, new, q)
    held_to_the_oracle(cache, new, q, o, lse, rows_each=12)


# ------------------------------------------------------------------ items of many steps

LONG_ITEMS = [  # D, window, sinks: pairs that are not cut, of 33 and more steps, and of 65 and more
    (64, 0, 0), (128, 0, 0), (64, 4500, 300), (128, 4500, 300), (128, 8200, 0),
]


@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", LONG_ITEMS)
def test_items_of_many_steps(dev, case, kept):
    """8400 tokens of 3 ranks with 8 query heads to a key head: 263 pairs of tiles for each rank, of up to 66 steps, and with
    so many to deal none of them is cut."""
    D, window, sinks = case
    lengths, R = [8400], 3
    d = B.fo_paged_desc(8, 1, head_dim=D, R=R, page=64, cache=kept, window=window, sinks=sinks)
    cache = Kept(dev, d, lengths, draws(1, 1, D, lengths), draws(2, 1, D, lengths))
    q = queries(3, d, 8400)
    o, lse = attend(dev, cache, lengths, q)
    held_to_the_oracle(cache, lengths, q, o, lse, rows_each=80)


# ------------------------------------------------------------------ infinities and NaN

ODD = [  # lengths, new, heads_q, heads_k, D, page, window, sinks: up to 16 rows a key head
    ([40, 9, 300, 129], [4, 3, 4, 2], 8, 2, 128, 16, 0, 0),
    ([40, 9, 300, 700], [4, 3, 4, 2], 4, 1, 64, 32, 33, 3),
    ([200, 70], [2, 2], 5, 1, 128, 64, 5, 0),
    ([300, 33, 140, 2], [16, 9, 11, 2], 2, 2, 128, 16, 0, 0),
    ([600, 140], [8, 7], 2, 1, 64, 64, 100, 4),
    ([20000, 15000], [5, 16], 3, 3, 128, 256, 0, 0),
    ([5, 16], [5, 16], 1, 1, 64, 32, 3, 1),
]


@pytest.mark.parametrize("where", ["new", "anywhere"])
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", ODD)
def test_values_that_are_no_numbers_reach_the_rows_that_see_them_alone(dev, case, kept, where):
    """Single elements of values (NaN; with bf16 infinities), an 8-bit token's scale, and keys: of new tokens, which the ones
    before them do not see, or of any."""
    lengths, new, hq, hk, D, page, window, sinks = case
    R = 2
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache=kept, window=window, sinks=sinks)
    cache = Kept(dev, d, lengths, draws(1, hk, D, lengths), draws(2, hk, D, lengths))
    g = np.random.default_rng(5)
    table = cache.table.cpu().numpy()
    for b, (n, m) in enumerate(zip(lengths, new)):
        pg, slot = P.places(table[b], n, page)
        for r in range(R):
            for what in ["nan", "inf", "-inf", "scale", "key"] * 2:
                j, h, e = int(g.integers(n - m if where == "new" else 0, n)), int(g.integers(hk)), int(g.integers(D))
                if what in ("scale", "key"):               # (of the last token, so that other rows stay clean)
                    j = n - 1
                if what == "key":
                    cache.kc[r][int(pg[j]), h, int(slot[j]), e] = NAN
                    cache.k[r][b][j, h, e] = NAN
                elif what == "scale":
                    if kept == "e4m3":
                        cache.vs[r][int(pg[j]), h, int(slot[j])] = float("inf")
                        with np.errstate(invalid="ignore"):
                            cache.v[r][b][j, h] = cache.v[r][b][j, h] * np.inf
                else:
                    value = NAN if kept == "e4m3" else float(what)
                    cache.vc[r][int(pg[j]), h, int(slot[j]), e] = value
                    cache.v[r][b][j, h, e] = value
    q = queries(3, d, sum(new))
    o, lse = attend(dev, cache, new, q)
    at, clean = 0, 0
    for b, (n, m) in enumerate(zip(lengths, new)):
        seen = P.sees(n, m, window, sinks)
        for r in range(R):
            k, v = cache.k[r][b], cache.v[r][b]
            for i in range(m):
                mine, p = f64(q[r][at + i]).reshape(1, hq, D), n - m + i
                with np.errstate(invalid="ignore", over="ignore"):
                    want, wl, size, far = (x[0] for x in P.attention(mine, k[:p + 1], v[:p + 1], 1, window, sinks))
                got, gl = o[r][at + i].reshape(hq, D), lse[r][at + i]
                fine = np.isfinite(want)
                assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (b, r, i)
                assert np.all(np.isfinite(got[fine])) and np.array_equal(np.isfinite(gl), np.isfinite(wl)), (b, r, i)
                rows = np.isfinite(wl)
                top = np.where(np.isfinite(v), np.abs(v), 0)[seen.any(axis=0)].max()
                score = (D + 8) * U * np.where(rows, far, 0)[:, None] + 2.0 ** -22
                bound = (2.0 ** -8 + 2 * score + (2 * n + 8) * U) * np.where(fine, size, 0) + n * 2.0 ** -31 * top + \
                    2.0 ** -8 * np.where(fine, np.abs(want), 0) * (1 + 2.0 ** -7)
                assert np.all(np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)) <= bound), (b, r, i)
                clean += int(fine.sum())
        at += m
    assert 0 < clean < R * sum(new) * hq * D                # (rows see some of them, and others none)

