"""CPU tests of the operators between the residual stream and the attention: the oracle pinned to known values and
to differences, and every refusal of the C ABI and the binding (no GPU needed: arguments are checked before the
device is looked at)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from oracle import layer_ops as O


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


# ------------------------------------------------------------------ the oracle

def test_e4m3_rounding_is_the_types_own():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = every[np.isfinite(every)]
    assert np.array_equal(O.round_e4m3(every), every) and every.max() == O.E4M3_TOP
    g = np.random.default_rng(0)
    v = np.concatenate([g.standard_normal(4000) * 10.0 ** g.uniform(-4, 2.6, 4000), [0.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625]])
    v = v[np.abs(v) <= 448].astype(np.float32)
    assert np.array_equal(O.round_e4m3(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_norm_gradient_matches_differences():
    g = np.random.default_rng(1)
    x, res, w, dy, dh = g.standard_normal((3, 7)), g.standard_normal((3, 7)), g.standard_normal(7), \
        g.standard_normal((3, 7)), g.standard_normal((3, 7))

    def loss(x, w):
        s, n, _ = O.rmsnorm(x, res, w, 1e-3, 1.0)
        return np.sum(n * dy) + np.sum(s * dh)

    s, _, rstd = O.rmsnorm(x, res, w, 1e-3, 1.0)
    dx, dw = O.rmsnorm_bwd(dy, dh, s, w, rstd, 1.0)
    d = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = d
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * d) - dx[i]) < 1e-7
    for i in range(7):
        e = np.zeros_like(w)
        e[i] = d
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * d) - dw[i]) < 1e-7


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(layout):
    g = np.random.default_rng(2)
    f, factor = O.rope_frequencies(6, 10000.0, "parts", 4.0, 64, 1.0, 8.0)
    x, dy = g.standard_normal((5, 16)), g.standard_normal((5, 16))
    pos = np.array([0, 1, -3, 1000, 77])
    # The map is linear: <dy, rope(x)> = <rope^T(dy), x>.
    y = O.rope(x, pos, f, factor, 8, layout)
    dx = O.rope(dy, pos, f, factor, 8, layout, inverse=True)
    assert abs(np.sum(y * dy) - np.sum(dx * x)) < 1e-12
    back = O.rope(y, pos, f, factor, 8, layout, inverse=True).reshape(5, 2, 8)
    want = x.reshape(5, 2, 8)
    assert np.allclose(back[..., :6], want[..., :6] * factor ** 2, atol=1e-12)
    assert np.array_equal(back[..., 6:], want[..., 6:])


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", stretch=4.0),
                                dict(scaling="wavelength", stretch=8.0, trained=8192, slow=1.0, fast=4.0),
                                dict(scaling="parts", stretch=16.0, trained=4096, slow=1.0, fast=32.0),
                                dict(scaling="parts", stretch=2.0, trained=2, slow=1.0, fast=32.0)])
@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (2, 1.5), (10, 1e6)])
def test_rope_frequencies_match_the_oracle(kw, rot, base):
    d = B.fo_rope_desc(128, 1, rot_dim=rot, base=base, **kw)
    f, factor = O.rope_frequencies(rot, base, **kw)
    got = np.array([d.turns[i] for i in range(rot // 2)], dtype=np.float64) * 2.0 ** -64 * 2 * math.pi
    # pow, the division by 2 pi and the mix: a few roundings of 2^-53 each, the fixed point's last place 2^-64.
    assert np.all(np.abs(got - f) <= 16 * 2.0 ** -53 * f + 2.0 ** -61)
    assert d.factor == pytest.approx(factor, rel=2.0 ** -23) and d.ready == 1


# ------------------------------------------------------------------ refusals

def code_of(f, *a, **k):
    with pytest.raises(B.FlashOverlapError) as e:
        f(*a, **k)
    return e.value.code


def norm_desc(**kw):
    d = B.fo_norm_desc(kw.pop("H", 256), R=kw.pop("R", 1))
    for k, v in kw.items():
        if k == "reserved":
            d.reserved[1] = v
        else:
            setattr(d, k, v)
    return d


BAD_NORM = [(dict(R=0), B.FO_ERR_INVALID_ARG), (dict(R=17), B.FO_ERR_INVALID_ARG), (dict(reserved=1), B.FO_ERR_INVALID_ARG),
            (dict(H=0), B.FO_ERR_SHAPE), (dict(H=B.FO_NORM_MAX_H + 1), B.FO_ERR_SHAPE), (dict(dtype=2), B.FO_ERR_DTYPE),
            (dict(w_dtype=-1), B.FO_ERR_DTYPE), (dict(eps=-1.0), B.FO_ERR_INVALID_ARG),
            (dict(eps=float("nan")), B.FO_ERR_INVALID_ARG), (dict(w_offset=float("nan")), B.FO_ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,code", BAD_NORM)
def test_norm_refuses_bad_descriptions(kw, code):
    d = norm_desc(**kw)
    lib = B.load()
    arr = (ctypes.c_void_p * 17)(*[256] * 17)
    assert lib.fo_rmsnorm(d, 4, arr, None, 256, arr, None, None, None, None, None) == code
    assert lib.fo_rmsnorm_bwd(d, 4, arr, None, arr, 256, arr, arr, None, None, None) == code
    size = ctypes.c_size_t()
    assert lib.fo_rmsnorm_bwd_workspace(d, 4, ctypes.byref(size)) == code


def test_norm_refuses_bad_pointers():
    d = B.fo_norm_desc(256, R=2)
    ok = [256, 512]
    call = lambda **k: code_of(B.fo_rmsnorm, d, k.pop("rows", 4), **{**dict(x=ok, residual=None, weight=256, h=ok, stream=0), **k})  # noqa: E731
    assert call(rows=-1) == B.FO_ERR_SHAPE
    assert call(x=[256, 0]) == B.FO_ERR_INVALID_ARG
    assert call(x=[256, 513]) == B.FO_ERR_ALIGN
    assert call(weight=0) == B.FO_ERR_INVALID_ARG
    assert call(weight=257) == B.FO_ERR_ALIGN
    assert call(h=None) == B.FO_ERR_INVALID_ARG          # nothing to write
    assert call(q=ok) == B.FO_ERR_INVALID_ARG            # values without their scales
    assert call(scale=ok) == B.FO_ERR_INVALID_ARG
    assert call(rstd=[256, 514]) == B.FO_ERR_ALIGN
    back = lambda **k: code_of(B.fo_rmsnorm_bwd, d, 4, **{**dict(dy=ok, dh=None, h=ok, weight=256, rstd=ok, dx=ok, stream=0), **k})  # noqa: E731
    assert back(dweight=256) == B.FO_ERR_INVALID_ARG     # no workspace
    assert back(dweight=256, ws=264) == B.FO_ERR_ALIGN
    assert back(dx=[256, 0]) == B.FO_ERR_INVALID_ARG
    assert back(dh=[256, 511]) == B.FO_ERR_ALIGN


def test_quant_refuses_bad_arguments():
    ok = [256]
    call = lambda rows=4, cols=128, x=ok, q=ok, s=ok, **k: code_of(B.fo_quant_fp8, rows, cols, x, q, s, **{**dict(dtype="bf16", stream=0), **k})  # noqa: E731
    assert call(rows=-1) == B.FO_ERR_SHAPE
    assert call(cols=0) == B.FO_ERR_SHAPE
    assert call(rows=2 ** 31) == call(rows=65535 * 128 + 1, block_rows=128) == B.FO_ERR_SHAPE
    assert call(block_rows=64) == B.FO_ERR_INVALID_ARG
    assert call(qt=ok, scale_t=ok) == B.FO_ERR_INVALID_ARG               # only blocks of 128 rows
    assert call(qt=ok, block_rows=128) == B.FO_ERR_INVALID_ARG
    assert call(x=[0]) == B.FO_ERR_INVALID_ARG
    assert call(x=[257]) == B.FO_ERR_ALIGN
    assert call(s=[258]) == B.FO_ERR_ALIGN
    assert B.load().fo_quant_fp8(1, 4, 4, 3, 1, None, None, None, None, None, None) == B.FO_ERR_DTYPE
    assert B.load().fo_quant_fp8(0, 4, 4, 0, 1, None, None, None, None, None, None) == B.FO_ERR_INVALID_ARG


def test_gemm_fp8_refuses_bad_arguments():
    ok = [256]

    def call(M=4, N=64, K=128, ws=256, R=1, reserved=0, out=0, **k):
        d = B.fo_gemm_fp8_desc(N, K)
        d.R, d.reserved[2], d.out_dtype = R, reserved, out
        a = dict(A=ok, sA=ok, W=ok, sW=ok, Y=ok)
        a.update(k)
        arr = [None if a[n] is None else (ctypes.c_void_p * 17)(*(a[n] * 17)[:17]) for n in ("A", "sA", "W", "sW", "Y")]
        return B.load().fo_gemm_fp8(d, M, *arr, ws, None)

    assert call(M=-1) == call(N=0) == call(K=0) == B.FO_ERR_SHAPE
    assert call(K=120) == B.FO_ERR_ALIGN
    assert call(R=0) == call(R=17) == call(reserved=1) == call(ws=0) == B.FO_ERR_INVALID_ARG
    assert call(ws=264) == B.FO_ERR_ALIGN
    assert call(out=7) == B.FO_ERR_DTYPE
    for name in ("A", "W", "Y"):
        assert call(**{name: [264]}) == B.FO_ERR_ALIGN
        assert call(**{name: [0]}) == call(**{name: None}) == B.FO_ERR_INVALID_ARG
    assert call(sA=[258]) == B.FO_ERR_ALIGN
    assert call(M=0) == B.FO_OK
    assert B.load().fo_ops_workspace_init(256, 8, None) == B.FO_ERR_INVALID_ARG
    assert B.load().fo_ops_workspace_init(None, 64, None) == B.FO_ERR_INVALID_ARG
    assert B.load().fo_ops_status_query(None, None, None) == B.FO_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), B.FO_ERR_INVALID_ARG), (dict(rot_dim=3), B.FO_ERR_SHAPE), (dict(rot_dim=130), B.FO_ERR_SHAPE),
    (dict(rot_dim=0), B.FO_ERR_SHAPE), (dict(base=1.0), B.FO_ERR_INVALID_ARG), (dict(base=float("nan")), B.FO_ERR_INVALID_ARG),
    (dict(scaling="linear", stretch=0.5), B.FO_ERR_INVALID_ARG), (dict(scaling="linear", stretch=float("inf")), B.FO_ERR_INVALID_ARG),
    (dict(scaling="wavelength", stretch=2.0, trained=0.0, slow=1.0, fast=4.0), B.FO_ERR_INVALID_ARG),
    (dict(scaling="parts", stretch=2.0, trained=64, slow=4.0, fast=4.0), B.FO_ERR_INVALID_ARG),
    (dict(scaling="parts", stretch=2.0, trained=64, slow=0.0, fast=4.0), B.FO_ERR_INVALID_ARG)])
def test_rope_refuses_bad_descriptions(kw, code):
    assert code_of(B.fo_rope_desc, 128, 2, 1, 1, **kw) == code


def test_rope_refuses_bad_arguments():
    assert code_of(B.fo_rope_desc, 257, 1) == code_of(B.fo_rope_desc, 128, 0) == code_of(B.fo_rope_desc, 128, 1, -1) == B.FO_ERR_SHAPE
    d = B.fo_rope_desc(128, 2, 1, 1)
    ok = [256]
    call = lambda rows=4, pos=256, q=ok, k=ok, v=ok, qo=ok, ko=ok, vo=ok, d=d: code_of(B.fo_rope, d, rows, pos, q, k, v, qo, ko, vo, stream=0)  # noqa: E731
    assert call(rows=-1) == B.FO_ERR_SHAPE
    assert call(q=[0]) == call(vo=[0]) == B.FO_ERR_INVALID_ARG
    assert call(k=[257]) == call(pos=260) == B.FO_ERR_ALIGN
    raw = B.RopeDesc()
    raw.R = raw.heads_q = 1
    raw.head_dim = raw.rot_dim = 128
    assert call(d=raw, k=None, v=None, ko=None, vo=None) == B.FO_ERR_INVALID_ARG      # fo_rope_init was not called
    one = (ctypes.c_void_p * 1)(256)
    ld, short = (ctypes.c_int64 * 3)(256, 128, 128), (ctypes.c_int64 * 3)(256, 127, 128)
    raw_call = lambda pos_bytes, li, lo, inv: B.load().fo_rope(d, 4, 256, pos_bytes, one, one, one, li, one, one, one, lo, inv, None)  # noqa: E731
    assert raw_call(2, ld, ld, 0) == raw_call(8, ld, ld, 2) == raw_call(8, None, ld, 0) == B.FO_ERR_INVALID_ARG
    assert raw_call(8, short, ld, 0) == raw_call(8, ld, short, 0) == B.FO_ERR_SHAPE


def test_binding_refuses_wrong_tensors():
    d = B.fo_norm_desc(256)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.fo_rmsnorm(d, 4, [x], None, w, [x], stream=0)
    with pytest.raises(ValueError, match="expected"):
        B.fo_rmsnorm(d, 5, [x], None, w, [x], stream=0)
    with pytest.raises(ValueError, match="expected"):
        B.fo_rmsnorm(d, 4, [x.float()], None, w, [x], stream=0)
    with pytest.raises(ValueError, match="ranks"):
        B.fo_rmsnorm(d, 4, [x, x], None, w, [x], stream=0)
    r = B.fo_rope_desc(128, 2)
    with pytest.raises(ValueError, match="dense"):
        B.fo_rope(r, 4, None, [torch.zeros(4, 512, dtype=torch.bfloat16)[:, ::2]], None, None, [x], None, None, stream=0)
    with pytest.raises(ValueError, match="positions"):
        B.fo_rope(r, 4, torch.zeros(4), [256], None, None, [256], None, None, stream=0)


def test_zero_rows_are_fine():
    B.fo_rmsnorm(B.fo_norm_desc(256), 0, [256], None, 256, [256], stream=0)
    B.fo_quant_fp8(0, 128, [256], [256], [256], dtype="f32", stream=0)
    B.fo_rope(B.fo_rope_desc(128, 2), 0, None, [256], None, None, [256], None, None, stream=0)


def test_calls_without_a_gpu_fail_loudly():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    no_gpu = (B.FO_ERR_CUDA, B.FO_ERR_UNSUPPORTED)
    assert code_of(B.fo_rmsnorm, B.fo_norm_desc(256), 4, [256], None, 256, [256], stream=0) in no_gpu
    assert code_of(B.fo_quant_fp8, 4, 128, [256], [256], [256], dtype="bf16", stream=0) in no_gpu
    assert code_of(B.fo_gemm_fp8, B.fo_gemm_fp8_desc(64, 128), 4, [256], [256], [256], [256], [256], 256, stream=0) in no_gpu
    assert code_of(B.fo_rope, B.fo_rope_desc(128, 2), 4, None, [256], None, None, [256], None, None, stream=0) in no_gpu
