"""RMSNorm with the residual's addition, its gradient, and quantisation to 8 bits, against the fp64 oracle.

Tolerances. u = 2^-24 is fp32's half step. A row's sum of H terms runs in fp32 as a per-thread sum of at most 64
terms and a tree over the threads: fewer than 80 roundings on any path, so the mean square is off by 80 u
relative (its terms are positive), rstd by half that and a few u: 44 u; a normed value by 48 u relative. A value stored in
type t adds half a step of t: eps(t)/2 relative. An 8-bit value times its scale is off by 2^-4 relative (e4m3's half
step) or, below the smallest normal 2^-6, by half a step 2^-10 of the scale. In the gradient, the sum of u h is
off by 80 u times the sum of magnitudes; the weight's gradient adds at most rows terms one after another.
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
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a GB300"
    return torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


def draw(g, rows, cols, dtype, dev, scale=1.0):
    return (torch.randn(rows, cols, generator=g) * scale).to(TYPES[dtype]).to(dev)


def empty(dev, *shape, dtype=torch.float32):
    # Poisoned, so that a value that is not written shows.
    t = torch.empty(shape, dtype=dtype, device=dev)
    return t.view(torch.uint8).fill_(0x7F).view(dtype) if t.numel() else t


def check_8_bits(q, scale, n, rel, up=1):
    """q (8 bits) and scale against the fp64 values n, known to `rel` relative."""
    want = O.block_scales(n, up)
    assert np.all(np.abs(f64(scale) - want) <= (rel + 2 * U) * want)
    each = O.spread(f64(scale), n.shape, up)
    got = f64(q)
    assert np.all(np.abs(got * each - n) <= 2.0 ** -4 * np.abs(n) * (1 + 1e-5) + 2.0 ** -10 * each + 4 * rel * np.abs(n))
    # Away from the borders between two 8-bit values, the very value.
    lo, hi = O.round_e4m3(n / each * (1 - 2 * rel - 4 * U)), O.round_e4m3(n / each * (1 + 2 * rel + 4 * U))
    assert np.all((got == lo) | (got == hi))


CASES = [(1, 1), (3, 7), (2, 128), (5, 129), (1, 4096), (7, 1000), (33, 256), (4, 2880), (3, 5120), (2, 8192), (3, 8200),
         (2, 16384), (1, 32768), (2, 32767), (3, 1357), (300, 512), (1000, 64), (700, 1024), (4000, 128), (2500, 9), (400, 4096)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,H", CASES)
def test_rmsnorm(dev, rows, H, residual, dtype):
    g = torch.Generator().manual_seed(rows * 7 + H)
    x, w = draw(g, rows, H, dtype, dev), (1 + 0.2 * torch.randn(H, generator=g)).to(TYPES[dtype]).to(dev)
    res = draw(g, rows, H, dtype, dev) if residual else None
    t = TYPES[dtype]
    h, y, q = empty(dev, rows, H, dtype=t), empty(dev, rows, H, dtype=t), empty(dev, rows, H, dtype=E4M3)
    scale, rstd = empty(dev, rows, -(-H // 128)), empty(dev, rows)
    B.fo_rmsnorm(B.fo_norm_desc(H, dtype=dtype, eps=1e-5), rows, [x], [res] if residual else None, w, [h], [y], [q],
                 [scale], [rstd])
    s, n, r = O.rmsnorm(f64(x), f64(res) if residual else None, f64(w), 1e-5)
    assert np.all(np.abs(f64(h) - s) <= (HALF[dtype] + U) * np.abs(s) * (1 + U))
    assert np.all(np.abs(f64(rstd) - r) <= 44 * U * r)
    assert np.all(np.abs(f64(y) - n) <= (HALF[dtype] + 48 * U) * np.abs(n) * (1 + 2.0 ** -7))
    check_8_bits(q, scale, n, 48 * U)


@pytest.mark.parametrize("outs", ["h", "y", "q", "r", "hq"])
def test_rmsnorm_writes_what_is_asked(dev, outs):
    g = torch.Generator().manual_seed(5)
    rows, H = 6, 384
    x, res, w = draw(g, rows, H, "bf16", dev), draw(g, rows, H, "bf16", dev), draw(g, 1, H, "f32", dev).view(H)
    h, y, q = (empty(dev, rows, H, dtype=t) for t in (torch.bfloat16, torch.bfloat16, E4M3))
    scale, rstd = empty(dev, rows, 3), empty(dev, rows)
    d = B.fo_norm_desc(H, w_dtype="f32", w_offset=1.0)
    has = lambda k, v: [v] if k in outs else None  # noqa: E731
    B.fo_rmsnorm(d, rows, [x], [res], w, has("h", h), has("y", y), has("q", q), has("q", scale), has("r", rstd))
    s, n, r = O.rmsnorm(f64(x), f64(res), f64(w), 1e-6, 1.0)
    if "h" in outs:
        assert np.all(np.abs(f64(h) - s) <= (2.0 ** -8 + U) * np.abs(s))
    if "y" in outs:
        assert np.all(np.abs(f64(y) - n) <= (2.0 ** -8 + 50 * U) * np.abs(n) * (1 + 2.0 ** -7))
    if "q" in outs:
        check_8_bits(q, scale, n, 50 * U)
    if "r" in outs:
        assert np.all(np.abs(f64(rstd) - r) <= 44 * U * r)


def test_rmsnorm_shards_alias_and_unaligned_rows(dev):
    # Three shards in one call, the sum written over the residual; then with a shard that starts off the 16-byte grid.
    g = torch.Generator().manual_seed(6)
    rows, H = 5, 256
    d = B.fo_norm_desc(H, R=3)
    w = draw(g, 1, H, "bf16", dev).view(H)
    buf = torch.zeros(rows * H + 1, dtype=torch.bfloat16, device=dev)
    x = [draw(g, rows, H, "bf16", dev) for _ in range(2)] + [buf[1:].view(rows, H)]
    x[2].copy_(draw(g, rows, H, "bf16", dev))
    for use in ([x[0], x[1], x[2].clone()], x):
        res = [draw(g, rows, H, "bf16", dev) for _ in range(3)]
        before = [f64(t) for t in res]
        y = [empty(dev, rows, H, dtype=torch.bfloat16) for _ in range(3)]
        B.fo_rmsnorm(d, rows, use, res, w, res, y)
        for r in range(3):
            s, n, _ = O.rmsnorm(f64(use[r]), before[r], f64(w), 1e-6)
            assert np.all(np.abs(f64(res[r]) - s) <= (2.0 ** -8 + U) * np.abs(s))
            assert np.all(np.abs(f64(y[r]) - n) <= (2.0 ** -8 + 50 * U) * np.abs(n) * (1 + 2.0 ** -7))


@pytest.mark.parametrize("H", [256, 1000, 131])
def test_rmsnorm_special_values_stay_in_their_row(dev, H):
    g = torch.Generator().manual_seed(7)
    x = torch.randn(5, H, generator=g)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, H - 1] = float("inf")
    x = x.to(dev)
    w = torch.ones(H, device=dev)
    y, q, scale = empty(dev, 5, H), empty(dev, 5, H, dtype=E4M3), empty(dev, 5, -(-H // 128))
    B.fo_rmsnorm(B.fo_norm_desc(H, dtype="f32"), 5, [x], None, w, None, [y], [q], [scale])
    y, q, scale = f64(y), f64(q), f64(scale)
    assert np.all(y[1] == 0) and np.all(q[1] == 0) and np.all(scale[1] == 2.0 ** -126)
    assert np.all(np.isnan(y[2])) and np.all(np.isnan(q[2])) and np.all(np.isnan(scale[2]))
    assert np.isnan(y[3, H - 1]) and np.isnan(scale[3, (H - 1) // 128])
    assert np.all(np.delete(y[3], H - 1) == 0)
    for row in (0, 4):
        _, n, _ = O.rmsnorm(f64(x)[row:row + 1], None, np.ones(H), 1e-6)
        assert np.all(np.abs(y[row] - n[0]) <= 50 * U * np.abs(n[0]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,H", CASES)
def test_rmsnorm_bwd(dev, rows, H, residual, dtype):
    g = torch.Generator().manual_seed(rows * 11 + H)
    t = TYPES[dtype]
    dy, h = draw(g, rows, H, dtype, dev), draw(g, rows, H, dtype, dev, 2.0)
    dh = draw(g, rows, H, dtype, dev) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(t).to(dev)
    _, _, r = O.rmsnorm(f64(h), None, f64(w), 1e-5)
    rstd = torch.from_numpy(r).float().to(dev)
    dx, dw = empty(dev, rows, H, dtype=t), empty(dev, H)
    d = B.fo_norm_desc(H, dtype=dtype, eps=1e-5)
    ws = torch.empty(B.fo_rmsnorm_bwd_workspace(d, rows), dtype=torch.uint8, device=dev)
    B.fo_rmsnorm_bwd(d, rows, [dy], [dh] if residual else None, [h], w, [rstd], [dx], dw, ws)
    r = f64(rstd)
    want_x, want_w = O.rmsnorm_bwd(f64(dy), f64(dh) if residual else None, f64(h), f64(w), r)
    uh = np.abs(f64(dy) * f64(w) * f64(h))
    a = np.abs(r[:, None] * f64(dy) * f64(w))
    b = np.abs(f64(h)) * (r ** 3 * np.mean(uh, axis=1))[:, None]
    c = np.abs(f64(dh)) if residual else 0.0
    assert np.all(np.abs(f64(dx) - want_x) <= HALF[dtype] * np.abs(want_x) * (1 + 2.0 ** -7) + 4 * U * (a + c) + 90 * U * b)
    assert np.all(np.abs(f64(dw) - want_w) <= (min(rows, 2000) + 4) * U * np.sum(np.abs(f64(dy) * f64(h) * r[:, None]), axis=0))


def test_rmsnorm_bwd_shards_repeat_and_need_no_weight_gradient(dev):
    g = torch.Generator().manual_seed(9)
    rows, H, R = 40, 512, 4
    d = B.fo_norm_desc(H, R=R, w_offset=1.0)
    make = lambda: [draw(g, rows, H, "bf16", dev) for _ in range(R)]  # noqa: E731
    dy, dh, h = make(), make(), make()
    w = draw(g, 1, H, "bf16", dev).view(H)
    rstd = [torch.rsqrt(t.float().square().mean(dim=1) + 1e-6) for t in h]
    ws = torch.empty(B.fo_rmsnorm_bwd_workspace(d, rows), dtype=torch.uint8, device=dev)
    runs = []
    for _ in range(2):
        ws.fill_(0x7F)
        dx, dw = [empty(dev, rows, H, dtype=torch.bfloat16) for _ in range(R)], empty(dev, H)
        B.fo_rmsnorm_bwd(d, rows, dy, dh, h, w, rstd, dx, dw, ws)
        runs.append((dx, dw))
    for a, b in zip(runs[0][0] + [runs[0][1]], runs[1][0] + [runs[1][1]]):
        assert torch.equal(a, b)
    alone = [empty(dev, rows, H, dtype=torch.bfloat16) for _ in range(R)]
    B.fo_rmsnorm_bwd(d, rows, dy, dh, h, w, rstd, alone)
    # In place over the upstream gradient of the residual.
    over = [t.clone() for t in dh]
    B.fo_rmsnorm_bwd(d, rows, dy, over, h, w, rstd, over)
    want = np.zeros(H)
    size = np.zeros(H)
    for r in range(R):
        assert torch.equal(alone[r], runs[0][0][r]) and torch.equal(over[r], alone[r])
        _, part = O.rmsnorm_bwd(f64(dy[r]), f64(dh[r]), f64(h[r]), f64(w), f64(rstd[r]), 1.0)
        want += part
        size += np.sum(np.abs(f64(dy[r]) * f64(h[r]) * f64(rstd[r])[:, None]), axis=0)
    assert np.all(np.abs(f64(runs[0][1]) - want) <= (R * rows + 4) * U * size)
    none = [t[:0] for t in dy]
    B.fo_rmsnorm_bwd(d, 0, none, none, none, w, [t[:0] for t in rstd], none, runs[0][1], ws)      # no rows: an empty sum
    assert torch.count_nonzero(runs[0][1]).item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 128), (5, 130), (257, 4096), (2, 100000), (64, 1357), (1, 16)])
def test_quant_rows(dev, rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = draw(g, rows, cols, dtype, dev, 30.0)
    q, scale = empty(dev, rows, cols, dtype=E4M3), empty(dev, rows, -(-cols // 128))
    B.fo_quant_fp8(rows, cols, [x], [q], [scale])
    check_8_bits(q, scale, f64(x), 2 * U)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 128), (129, 257), (1000, 144), (384, 4096), (50, 1357), (300, 16), (1001, 264), (131, 128), (2, 8),
                                       (130, 1000)])
@pytest.mark.parametrize("transposed", [False, True])
def test_quant_blocks(dev, rows, cols, dtype, transposed):
    g = torch.Generator().manual_seed(rows + cols)
    x = [draw(g, rows, cols, dtype, dev, 0.02) for _ in range(2)]
    up, across = -(-rows // 128), -(-cols // 128)
    q, scale = [empty(dev, rows, cols, dtype=E4M3) for _ in x], [empty(dev, up, across) for _ in x]
    qt, st = [empty(dev, cols, rows, dtype=E4M3) for _ in x], [empty(dev, across, up) for _ in x]
    B.fo_quant_fp8(rows, cols, x, q, scale, *((qt, st) if transposed else ()), block_rows=128)
    for r in range(2):
        check_8_bits(q[r], scale[r], f64(x[r]), 2 * U, up=128)
        if transposed:
            assert np.array_equal(f64(qt[r]), f64(q[r]).T) and torch.equal(st[r], scale[r].t())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant_special_values(dev, block_rows):
    x = torch.randn(256, 384)
    x[:128, 128:256] = 0
    x[130, 5] = float("inf")
    x[200, 300] = float("nan")
    x[3, 0] = 1e-45                                     # a group of the smallest magnitude: its scale is held up
    x[3, 1:128] = 0
    x = x.to(dev)
    q, scale = empty(dev, 256, 384, dtype=E4M3), empty(dev, 256 // block_rows, 3)
    B.fo_quant_fp8(256, 384, [x], [q], [scale], block_rows=block_rows)
    q, scale = f64(q), f64(scale)
    at = lambda row: row // block_rows  # noqa: E731
    assert scale[0, 1] == 2.0 ** -126 and np.all(q[0, 128:256] == 0)
    assert np.isinf(scale[at(130), 0]) and np.isnan(q[130, 5]) and q[130, 6] == 0
    assert np.isnan(scale[at(200), 2]) and np.all(np.isnan(q[200, 256:]))
    if block_rows == 1:
        assert scale[3, 0] == 2.0 ** -126
    assert np.all(np.isfinite(q[:128])) and np.all(np.isfinite(scale[at(127)]))


@pytest.mark.parametrize("at_q,at_t", [(0, 0), (8, 0), (0, 8), (8, 1), (1, 16), (0, 3)])
@pytest.mark.parametrize("rows,cols", [(272, 144), (16, 128), (400, 1040), (264, 256)])
def test_quant_blocks_outputs_off_the_wide_grid(dev, rows, cols, at_q, at_t):
    """The widths of the stores go by where rows and the copy's lines start; nothing beside them is touched."""
    g = torch.Generator().manual_seed(at_q + at_t)
    x = draw(g, rows, cols, "bf16", dev, 0.02)
    n, pad = rows * cols, 32
    qs, ts = (torch.full((n + 2 * pad,), 85, dtype=torch.uint8, device=dev) for _ in range(2))
    q, qt = qs[pad + at_q:][:n].view(rows, cols), ts[pad + at_t:][:n].view(cols, rows)
    scale, st = empty(dev, -(-rows // 128), -(-cols // 128)), empty(dev, -(-cols // 128), -(-rows // 128))
    B.fo_quant_fp8(rows, cols, [x], [q], [scale], [qt], [st], block_rows=128)
    check_8_bits(q.view(E4M3), scale, f64(x), 2 * U, up=128)
    assert torch.equal(qt, q.t()) and torch.equal(st, scale.t())
    for buf, at in ((qs, at_q), (ts, at_t)):
        assert (buf[:pad + at] == 85).all() and (buf[pad + at + n:] == 85).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [0, 1, 3, 6])
@pytest.mark.parametrize("rows,H", [(1, 1), (3, 5), (5, 257), (2, 255), (7, 1357), (3, 2050), (2, 4099), (2, 8193), (1, 20001)])
def test_norm_of_rows_that_start_anywhere(dev, rows, H, at, dtype):
    """Rows off the 16-byte grid, from any element of a larger buffer: the values of rows on it, forward and backward,
    and nothing beside the outputs is touched."""
    g = torch.Generator().manual_seed(rows + H + at)
    T, n, pad = TYPES[dtype], rows * H, 40
    d = B.fo_norm_desc(H, dtype=dtype)

    def inside(t):
        buf = torch.full((t.numel() + 2 * pad,), 7, dtype=t.dtype, device=dev)
        buf[pad + at:][:t.numel()] = t.reshape(-1)
        return buf, buf[pad + at:][:t.numel()].view(t.shape)

    x, res, dy, dh = (torch.randn(rows, H, generator=g).to(T).to(dev) for _ in range(4))
    w = (1 + torch.randn(H, generator=g)).to(T).to(dev)
    outs = {k: torch.zeros(rows, H, dtype=T, device=dev) for k in ("h", "y", "dx")}
    q, s, r = torch.zeros(rows, H, dtype=torch.uint8, device=dev), empty(dev, rows, -(-H // 128)), empty(dev, rows)
    dw, ws = empty(dev, H), torch.empty(B.fo_rmsnorm_bwd_workspace(d, rows), dtype=torch.uint8, device=dev)
    moved = {k: inside(v) for k, v in dict(outs, x=x, res=res, dy=dy, dh=dh, w=w, q=q).items()}
    m = {k: v[1] for k, v in moved.items()}
    B.fo_rmsnorm(d, rows, [m["x"]], [m["res"]], m["w"], [m["h"]], [m["y"]], [m["q"]], [s], [r])
    want_s, want_n, want_r = O.rmsnorm(f64(x), f64(res), f64(w), 1e-6)
    half = torch.finfo(T).eps / 2
    assert np.all(np.abs(f64(m["h"]) - want_s) <= (half + U) * np.abs(want_s))
    assert np.all(np.abs(f64(r) - want_r) <= 44 * U * want_r)
    assert np.all(np.abs(f64(m["y"]) - want_n) <= (half + 48 * U) * np.abs(want_n) * (1 + 2.0 ** -7))
    check_8_bits(m["q"].view(E4M3), s, want_n, 48 * U)
    B.fo_rmsnorm_bwd(d, rows, [m["dy"]], [m["dh"]], [m["h"]], m["w"], [r], [m["dx"]], dw, ws)
    hh, rr = m["h"].clone(), r.clone()
    dx2, dw2 = torch.zeros(rows, H, dtype=T, device=dev), empty(dev, H)
    B.fo_rmsnorm_bwd(d, rows, [dy], [dh], [hh], w, [rr], [dx2], dw2, ws)
    assert torch.equal(m["dx"], dx2) and torch.equal(dw, dw2)
    for k in ("h", "y", "dx", "q"):
        buf, t = moved[k]
        assert (buf[:pad + at] == 7).all() and (buf[pad + at + t.numel():] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("H", [512, 640, 1024, 1280, 1408, 2048, 2304, 4096, 4352, 5610, 6016, 8192, 8704, 8886, 16384])
def test_norm_backward_of_many_rows(dev, H, residual, dtype):
    """More rows than blocks, at every number of warps and chunks: each ring of rows goes round, and the same row
    gives the same gradient wherever it stands."""
    g = torch.Generator().manual_seed(H)
    T, few, times = TYPES[dtype], 7, 700
    dy, h, dh = (torch.randn(few, H, generator=g).to(T).to(dev) for _ in range(3))
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(T).to(dev)
    r = (0.5 + torch.rand(few, generator=g)).to(dev)
    d = B.fo_norm_desc(H, dtype=dtype)

    def run(n, dy, dh, h, r):
        dx, dw = empty(dev, n, H, dtype=T), empty(dev, H)
        ws = torch.empty(B.fo_rmsnorm_bwd_workspace(d, n), dtype=torch.uint8, device=dev)
        B.fo_rmsnorm_bwd(d, n, [dy], [dh] if residual else None, [h], w, [r], [dx], dw, ws)
        return dx, dw

    dx, dw = run(few, dy, dh, h, r)
    many = [t.repeat(times, *[1] * (t.dim() - 1)) for t in (dy, dh, h, r)]
    dx2, dw2 = run(few * times, *many)
    assert torch.equal(dx2, dx.repeat(times, 1))
    # Sums of 4900 terms against 700 times sums of 7 in fp32: 4900 roundings of the magnitudes' sum.
    size = (dy.double() * h.double() * r.double()[:, None]).abs().sum(dim=0) * times
    assert ((dw2.double() - times * dw.double()).abs() <= 4910 * U * size).all()
    want, _ = O.rmsnorm_bwd(f64(dy), f64(dh) if residual else None, f64(h), f64(w), f64(r))
    a = np.abs(f64(r)[:, None] * f64(dy) * f64(w))
    b = np.abs(f64(h)) * (f64(r) ** 3 * np.mean(np.abs(f64(dy) * f64(w) * f64(h)), axis=1))[:, None]
    c = np.abs(f64(dh)) if residual else 0.0
    assert np.all(np.abs(f64(dx) - want) <= HALF[dtype] * np.abs(want) * (1 + 2.0 ** -7) + 4 * U * (a + c) + 90 * U * b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [64, 128, 201, 256, 390, 512, 768, 1000, 1280, 2048])
def test_rmsnorm_of_many_rows(dev, H, dtype):
    """More rows than blocks: the same row gives the same values wherever it stands, on every shard."""
    g = torch.Generator().manual_seed(H)
    few, times, R = 9, 900, 2
    x, res = (draw(g, few, H, dtype, dev) for _ in range(2))
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(TYPES[dtype]).to(dev)
    d = B.fo_norm_desc(H, R=R, dtype=dtype)

    def run(n, x, res):
        outs = [[empty(dev, n, H, dtype=TYPES[dtype]) for _ in range(R)] for _ in range(2)]
        outs += [[empty(dev, n, H, dtype=torch.uint8) for _ in range(R)], [empty(dev, n, -(-H // 128)) for _ in range(R)],
                 [empty(dev, n) for _ in range(R)]]
        B.fo_rmsnorm(d, n, [x, res], [res, x], w, *outs)
        return outs

    for a, b in zip(run(few, x, res), run(few * times, x.repeat(times, 1), res.repeat(times, 1))):
        for s, m in zip(a, b):
            assert torch.equal(m, s.repeat(times, *[1] * (s.dim() - 1)))
