"""Rotary positions against the fp64 oracle.

Tolerance. The angle's fraction of a turn is exact but for the frequency's own rounding (2^-61 relative to a turn, times
the position); as fp32 half turns it is off by 2^-24 relative, at most pi 2^-24 in radians; sincospi adds up to 2 ulp, 2^-23,
and the factor and the two products half a step each: cos and sin count as off by 8 u (u = 2^-24), so a result by
8 u factor (|a| + |b|), and half a step of its type when it is stored.
"""
import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from oracle import layer_ops as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, x, pos, f, factor, D, layout, dtype, inverse):
    want = O.rope(x, pos, f, factor, D, layout, inverse)
    rows, rot = x.shape[0], 2 * len(f)
    v = np.abs(x.reshape(rows, -1, D))
    size = np.zeros_like(v)
    pairs = rot // 2
    ia = np.arange(pairs) if layout == "half" else 2 * np.arange(pairs)
    ib = ia + pairs if layout == "half" else ia + 1
    size[:, :, ia] = size[:, :, ib] = factor * (v[:, :, ia] + v[:, :, ib])
    # The frequency's rounding times the position, in radians: 16 * 2^-53 of the angle.
    far = 8 * U + 16 * 2.0 ** -53 * np.max(np.abs(pos)) if len(pos) else 0
    bound = far * size.reshape(rows, -1) + HALF[dtype] * np.abs(want) * (1 + 2.0 ** -7)
    bound.reshape(rows, -1, D)[:, :, rot:] = 0        # what is not rotated is copied
    assert np.all(np.abs(got - want) <= bound)


SHAPES = [(1, 1, 0, 0, 2, 2), (5, 2, 1, 1, 128, 128), (33, 4, 4, 4, 128, 64), (3, 8, 2, 2, 64, 64), (7, 3, 1, 0, 80, 20),
          (9, 2, 2, 1, 96, 48), (4, 1, 1, 1, 256, 256), (2, 5, 1, 1, 33, 6), (300, 2, 1, 1, 128, 128), (6, 2, 1, 2, 192, 48),
          (1, 32, 8, 8, 128, 128), (70, 1, 1, 1, 8, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("rows,hq,hk,hv,D,rot", SHAPES)
def test_rope_from_packed_rows_and_back(dev, rows, hq, hk, hv, D, rot, inverse, layout, dtype):
    g = torch.Generator().manual_seed(rows * 3 + D)
    R = 1 + rows % 3
    kw = dict(scaling="parts", stretch=8.0, trained=4096, slow=1.0, fast=32.0)
    d = B.fo_rope_desc(D, hq, hk, hv, R=R, rot_dim=rot, layout=layout, dtype=dtype, base=500000.0, **kw)
    f, factor = O.rope_frequencies(rot, 500000.0, **kw)
    pos = torch.randint(-5, 1 << 20, (rows,), generator=g, dtype=torch.int32 if rows % 2 else torch.int64)
    heads = (hq, hk, hv)
    packed = [torch.randn(rows, sum(heads) * D, generator=g).to(TYPES[dtype]).to(dev) for _ in range(R)]
    parts = [[p.split([n * D for n in heads], dim=1)[j] for p in packed] for j in range(3)]
    outs = [[torch.full((rows, n * D), float("nan"), dtype=TYPES[dtype], device=dev) for _ in range(R)] for n in heads]
    B.fo_rope(d, rows, pos.to(dev), *parts, *outs, inverse=inverse)
    for j in range(3):
        for r in range(R):
            if heads[j] and j < 2:
                check(f64(outs[j][r]), f64(parts[j][r]), pos.numpy().astype(np.float64), f, factor, D, layout, dtype, inverse)
            elif heads[j]:
                assert torch.equal(outs[j][r], parts[j][r])
    # Into packed rows (the gradient's way), and in place, give the same bits.
    back = [torch.full_like(p, float("nan")) for p in packed]
    to = [[p.split([n * D for n in heads], dim=1)[j] for p in back] for j in range(3)]
    B.fo_rope(d, rows, pos.to(dev), *[[t.contiguous() for t in p] for p in parts], *to, inverse=inverse)
    B.fo_rope(d, rows, pos.to(dev), *parts, *parts, inverse=inverse)
    for r in range(R):
        whole = torch.cat([outs[j][r] for j in range(3)], dim=1)
        assert torch.equal(back[r], whole) and torch.equal(packed[r], whole)


@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", stretch=4.0),
                                     dict(scaling="wavelength", stretch=8.0, trained=8192, slow=1.0, fast=4.0)])
def test_rope_far_positions_and_row_numbers(dev, scaling):
    # Positions beyond 2^24 (where fp32 has no whole numbers left), and none at all: the row's number.
    D, rows = 128, 64
    d = B.fo_rope_desc(D, 2, 1, dtype="f32", base=10000.0, **scaling)
    f, factor = O.rope_frequencies(D, 10000.0, **scaling)
    g = torch.Generator().manual_seed(3)
    q, k = torch.randn(rows, 2 * D, generator=g).to(dev), torch.randn(rows, D, generator=g).to(dev)
    for pos in (torch.arange(rows) * 7 + (1 << 27) + 1, None):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        B.fo_rope(d, rows, None if pos is None else pos.to(dev), [q], [k], None, [qo], [ko], None)
        at = (np.arange(rows) if pos is None else pos.numpy()).astype(np.float64)
        check(f64(qo), f64(q), at, f, factor, D, "half", "f32", False)
        check(f64(ko), f64(k), at, f, factor, D, "half", "f32", False)


def test_rope_leaves_what_lies_between_the_rows(dev):
    # Outputs that are parts of wider rows: the columns beside them are not touched; NaN and infinities stay in their pair.
    D, rows = 64, 9
    d = B.fo_rope_desc(D, 1, rot_dim=32)
    wide = torch.zeros(rows, 3 * D, dtype=torch.bfloat16, device=dev)
    x = torch.randn(rows, D).to(torch.bfloat16)
    x[2, 3], x[4, 40] = float("nan"), float("inf")
    B.fo_rope(d, rows, None, [x.to(dev)], None, None, [wide[:, D:2 * D]], None, None)
    got = f64(wide)
    assert np.all(got[:, :D] == 0) and np.all(got[:, 2 * D:] == 0)
    mid = got[:, D:2 * D]
    assert np.isnan(mid[2, 3]) and np.isnan(mid[2, 19]) and np.isinf(mid[4, 40])
    mid[2, [3, 19]] = 0
    mid[4, 40] = 0
    assert np.all(np.isfinite(mid))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_many_ranks_of_few_heads(dev, layout):
    # Threads that go through several ranks, the last of them through fewer.
    R, rows, D = 5, 16001, 64
    d = B.fo_rope_desc(D, 1, 1, R=R, layout=layout)
    f, factor = O.rope_frequencies(D, 10000.0)
    g = torch.Generator().manual_seed(4)
    q, k = ([torch.randn(rows, D, generator=g).to(torch.bfloat16).to(dev) for _ in range(R)] for _ in range(2))
    qo, ko = ([torch.full_like(t, float("nan")) for t in ts] for ts in (q, k))
    B.fo_rope(d, rows, None, q, k, None, qo, ko, None)
    at = np.arange(rows).astype(np.float64)
    for r in range(R):
        check(f64(qo[r]), f64(q[r]), at, f, factor, D, layout, "bf16", False)
        check(f64(ko[r]), f64(k[r]), at, f, factor, D, layout, "bf16", False)
