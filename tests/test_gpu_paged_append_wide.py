"""Appends to a paged cache that are large enough for a thread to go through many heads, or through several ranks', and
descriptions of rotary positions that are scaled, against the rotary call alone."""
import numpy as np
import pytest
import torch

import test_gpu_paged as T
from ag_gemm_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


MANY_HEADS = [  # as the operator's own cases; 628 and 640 blocks of tokens: a thread has all heads of a rank
    (4, 10, 5, 128, 64, 128, "half", [3000, 2100, 70], [2900, 2090, 35], 0),
    (4, 9, 3, 64, 16, 32, "interleaved", [9000, 1240], [9000, 1200], 4),
    (2, 6, 6, 128, 128, None, "half", [10100], [10100], 0),
]
MANY_RANKS = [  # fewer than eight heads a rank: a thread has two or four ranks', or what is left of them
    (16, 1, 1, 128, 64, 128, "half", [1500, 1200, 33], [1400, 1100, 33], 0),
    (13, 1, 1, 128, 32, 64, "interleaved", [3400], [3300], 4),
    (5, 2, 1, 64, 16, 64, "half", [16400], [16390], 0),
    (16, 2, 2, 64, 64, None, "half", [5200], [5100], 0),
]


@pytest.mark.parametrize("given", [None, torch.int32])
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", MANY_HEADS + MANY_RANKS)
def test_append_of_many_tokens(dev, case, kept, given):
    T.test_append(dev, case, kept, given)


SCALED = [dict(), dict(scaling="linear", stretch=4.0), dict(scaling="wavelength", stretch=8.0, trained=8192.0, slow=1.0, fast=4.0),
          dict(scaling="parts", stretch=16.0, trained=4096.0, slow=1.0, fast=32.0)]


@pytest.mark.parametrize("wide", [0, 8, 3])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("layout,rot", [("half", 128), ("interleaved", 64), ("half", 6)])
@pytest.mark.parametrize("scaled", SCALED)
def test_what_is_turned_is_what_the_rotary_call_turns(dev, scaled, layout, rot, given, wide):
    """Queries and a bf16 cache's keys, with scaled frequencies and the factor that comes with them: bit for bit what the
    rotary call makes of dense rows, wherever the append's rows lie. (Six turned values are not on the rotary call's
    16-byte grid, and its code for those rounds in another order: one step of bf16 at most.)"""
    hq, hk, D, R, page = 4, 2, 128, 2, 16
    lengths, new = [400, 33, 70], [100, 33, 1]
    rows = sum(new)
    rope = B.fo_rope_desc(D, hq, hk, hk, R=R, rot_dim=rot, layout=layout, base=10000.0, **scaled)
    assert (rope.factor != 1.0) == (scaled.get("scaling") == "parts")
    d = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page)
    cache = T.Cache(dev, d, lengths, [0] * 3, seed=3)
    cache.table, cache.new = torch.from_numpy(cache.table_all).to(dev), new
    g = torch.Generator().manual_seed(5)
    heads = (hq, hk, hk)
    packed = [torch.randn(rows, sum(heads) * D + wide, generator=g).to(BF).to(dev) for _ in range(R)]
    parts = [[p[:, :sum(heads) * D].split([n * D for n in heads], dim=1)[j] for p in packed] for j in range(3)]
    at = np.concatenate([np.arange(n - m, n) for n, m in zip(lengths, new)])
    pos = torch.randint(-5, 1 << 20, (rows,), generator=g).to(dev) if given else torch.from_numpy(at).to(dev)
    q_out = [torch.empty(rows, hq * D, dtype=BF, device=dev) for _ in range(R)]
    B.fo_kv_append(d, rope, cache.batch(dev), rows, *parts, q_out, cache.kc, cache.vc, positions=pos if given else None)
    out = [[torch.empty(rows, n * D, dtype=BF, device=dev) for _ in range(R)] for n in heads]
    B.fo_rope(rope, rows, pos, *[[x.contiguous() for x in xs] for xs in parts], *out)
    of = np.repeat(np.arange(3), new)
    page_of, slot = (torch.from_numpy(x.astype(np.int64)).to(dev) for x in (cache.table_all[of, at // page], at % page))
    for r in range(R):
        held = [c[page_of, :, slot].reshape(rows, hk * D) for c in (cache.kc[r], cache.vc[r])]
        for j, mine in enumerate([q_out[r]] + held):
            apart = (mine.view(torch.int16).int() - out[j][r].view(torch.int16).int()).abs().max().item()
            assert apart <= (1 if rot == 6 and j < 2 else 0)
