"""CPU tests of serving from a paged cache: the oracle pinned to softmax by hand and to a dense mask, and every refusal of
the C ABI and the binding (arguments are checked before the device is looked at)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from ag_gemm_gb300 import binding as B
from oracle import paged as P


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


# ------------------------------------------------------------------ the oracle

def test_sight():
    assert P.sees(5, 2, 0, 0).astype(int).tolist() == [[1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert P.sees(6, 2, 2, 1).astype(int).tolist() == [[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert P.sees(3, 1, 1, 0).astype(int).tolist() == [[0, 0, 1]]
    assert not P.sees(1, 3, 0, 0)[:2].any() and P.sees(1, 3, 0, 0)[2].all()
    page, slot = P.places([9, 4, 7], 5, 2)
    assert page.tolist() == [9, 9, 4, 4, 7] and slot.tolist() == [0, 1, 0, 1, 0]


def test_attention_is_softmax_under_a_dense_mask():
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((7, 2, 8)), g.standard_normal((7, 2, 8))
    o, lse, size, far = P.attention(q, k, v, 3, 3, 1, 0.5)
    mask = torch.from_numpy(P.sees(7, 3, 3, 1))
    for h in range(4):
        s = torch.from_numpy(q[:, h] @ k[:, h // 2].T * 0.5).masked_fill(~mask, -math.inf)
        assert np.allclose(o[:, h], (torch.softmax(s, 1) @ torch.from_numpy(v[:, h // 2])).numpy(), atol=1e-14)
        assert np.allclose(lse[:, h], torch.logsumexp(s, 1).numpy(), atol=1e-14)
    assert np.all(size >= np.abs(o) - 1e-15) and np.all(far >= 0)
    o, lse, _, _ = P.attention(q, k[:1], v[:1], 3, 0, 0)
    assert not o[:2].any() and np.all(lse[:2] == -math.inf) and np.allclose(o[2], v[0, [0, 0, 1, 1]])


def test_8_bits_of_a_head():
    x = np.array([[[0.0, 0.0], [-896.0, 448.0]]])
    q, s = P.in_8_bits(x)
    assert s.tolist() == [[2.0 ** -126, 2.0]] and q.tolist() == [[[0, 0], [-448, 224]]]


# ------------------------------------------------------------------ refusals

def desc(**kw):
    d = B.fo_paged_desc(8, 2, R=kw.pop("R", 1))
    for k, v in kw.items():
        if k == "reserved":
            d.reserved[2] = v
        else:
            setattr(d, k, v)
    return d


def batch(**kw):
    b = B.PagedBatch()
    b.seqs, b.max_new, b.pages, b.table_cols, b.lengths, b.starts, b.table = 3, 1, 10, 4, 256, None, 256
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def array(v):
    return None if v is None else (ctypes.c_void_p * 17)(*([v] * 17 if isinstance(v, int) else (v * 17)[:17]))


ARRAYS = ("q", "k", "v", "q_out", "k_cache", "v_cache", "k_scale", "v_scale")


def append(d=None, b=None, rows=3, rope=None, positions=None, pos_bytes=8, ld=(1024, 256, 256, 1024), ws=None, **k):
    a = {**dict.fromkeys(ARRAYS, 256), "k_scale": None, "v_scale": None, **k}
    x = {n: array(v) for n, v in a.items()}
    lds = None if ld is None else (ctypes.c_int64 * 4)(*ld)
    return B.load().fo_kv_append(d if d is not None else desc(), rope, b if b is not None else batch(), rows, positions, pos_bytes,
                                 x["q"], x["k"], x["v"], x["q_out"], lds, x["k_cache"], x["v_cache"], x["k_scale"], x["v_scale"], ws, None)


def attention(d=None, b=None, rows=3, ld=(1024, 1024), ws=256, **k):
    a = {**dict.fromkeys(("q", "k_cache", "v_cache", "o"), 256), "k_scale": None, "v_scale": None, "lse": None, **k}
    x = {n: array(v) for n, v in a.items()}
    lds = None if ld is None else (ctypes.c_int64 * 2)(*ld)
    return B.load().fo_paged_attention(d if d is not None else desc(), b if b is not None else batch(), rows, x["q"], lds, x["k_cache"],
                                       x["v_cache"], x["k_scale"], x["v_scale"], x["o"], x["lse"], ws, None)


BAD_DESC = [(dict(R=0), B.FO_ERR_INVALID_ARG), (dict(R=17), B.FO_ERR_INVALID_ARG), (dict(reserved=1), B.FO_ERR_INVALID_ARG),
            (dict(heads_q=0), B.FO_ERR_SHAPE), (dict(heads_k=0), B.FO_ERR_SHAPE), (dict(heads_q=9), B.FO_ERR_SHAPE),
            (dict(heads_q=130), B.FO_ERR_SHAPE), (dict(heads_k=-2), B.FO_ERR_SHAPE), (dict(head_dim=96), B.FO_ERR_SHAPE),
            (dict(head_dim=256), B.FO_ERR_SHAPE), (dict(page=8), B.FO_ERR_SHAPE), (dict(page=48), B.FO_ERR_SHAPE),
            (dict(page=512), B.FO_ERR_SHAPE), (dict(cache_dtype=2), B.FO_ERR_DTYPE), (dict(window=-1), B.FO_ERR_INVALID_ARG),
            (dict(sinks=-1), B.FO_ERR_INVALID_ARG), (dict(scale=-1.0), B.FO_ERR_INVALID_ARG),
            (dict(scale=float("nan")), B.FO_ERR_INVALID_ARG), (dict(scale=float("inf")), B.FO_ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_bad_descriptions_are_refused(kw, code):
    d = desc(**kw)
    size = ctypes.c_size_t()
    assert append(d) == attention(d) == B.load().fo_paged_attention_workspace(d, 1, 1, 1, ctypes.byref(size)) == code


BAD_BATCH = [(dict(seqs=-1), B.FO_ERR_SHAPE), (dict(seqs=4), B.FO_ERR_SHAPE), (dict(max_new=0), B.FO_ERR_SHAPE),
             (dict(max_new=2), B.FO_ERR_SHAPE), (dict(pages=0), B.FO_ERR_SHAPE), (dict(pages=2 ** 30), B.FO_ERR_SHAPE),
             (dict(table_cols=0), B.FO_ERR_SHAPE), (dict(table_cols=2 ** 25), B.FO_ERR_SHAPE), (dict(lengths=None), B.FO_ERR_INVALID_ARG),
             (dict(table=None), B.FO_ERR_INVALID_ARG), (dict(lengths=258), B.FO_ERR_ALIGN), (dict(table=257), B.FO_ERR_ALIGN),
             (dict(starts=258), B.FO_ERR_ALIGN)]


@pytest.mark.parametrize("kw,code", BAD_BATCH)
def test_bad_batches_are_refused(kw, code):
    assert append(b=batch(**kw)) == attention(b=batch(**kw)) == code


def test_as_many_entries_as_positions_have_numbers_for():
    for page in (16, 64, 256):
        most = 2 ** 30 // page
        for call in (append, attention):
            assert call(desc(page=page), batch(table_cols=most), q=[257]) == B.FO_ERR_ALIGN     # (what is checked next)
            assert call(desc(page=page), batch(table_cols=most + 1), q=[257]) == B.FO_ERR_SHAPE


def test_bad_arguments_are_refused():
    for call, names in ((append, ("q", "k", "v", "q_out", "k_cache", "v_cache")), (attention, ("q", "k_cache", "v_cache", "o"))):
        assert call(rows=-1) == call(rows=2 ** 31) == call(rows=2) == B.FO_ERR_SHAPE
        assert call(ld=None) == B.FO_ERR_INVALID_ARG
        assert call(ws=264) == B.FO_ERR_ALIGN
        for name in names:
            assert call(**{name: [0]}) == call(**{name: None}) == B.FO_ERR_INVALID_ARG
            assert call(**{name: [257]}) == B.FO_ERR_ALIGN
        assert call(k_cache=[264]) == call(v_cache=[264]) == B.FO_ERR_ALIGN
        # Scales belong to an 8-bit cache, and that to them.
        assert call(k_scale=256) == call(v_scale=256) == B.FO_ERR_INVALID_ARG
        eight = desc(cache_dtype=1)
        assert call(eight, k_scale=256) == call(eight, v_scale=256) == B.FO_ERR_INVALID_ARG
        assert call(eight, k_scale=256, v_scale=260) == B.FO_ERR_ALIGN
        # Nothing to do, whatever the pointers.
        none = dict.fromkeys(names)
        assert call(b=batch(seqs=0), **none) == B.FO_OK
        assert call(b=batch(starts=256, lengths=None), rows=0, **none) == B.FO_OK
        assert B.load().fo_paged_attention(None, batch(), 3, *[None] * 10) == B.FO_ERR_INVALID_ARG
        assert call(b=batch(starts=256), rows=2, q=None) == B.FO_ERR_INVALID_ARG
    assert attention(ws=None) == B.FO_ERR_INVALID_ARG
    assert attention(ld=(1016, 1024)) == attention(ld=(1024, 1016)) == B.FO_ERR_SHAPE
    assert attention(ld=(1028, 1024)) == attention(ld=(1024, 1028)) == B.FO_ERR_ALIGN
    assert attention(q=[264]) == attention(o=[264]) == attention(lse=[258]) == B.FO_ERR_ALIGN
    for i in range(4):
        ld = [1024, 256, 256, 1024]
        ld[i] -= 1
        assert append(ld=ld) == B.FO_ERR_SHAPE
    assert append(positions=256, pos_bytes=2) == B.FO_ERR_INVALID_ARG
    assert append(positions=260, pos_bytes=8) == append(positions=258, pos_bytes=4) == B.FO_ERR_ALIGN
    size = ctypes.c_size_t()
    w = B.load().fo_paged_attention_workspace
    assert w(desc(), 1, 1, 1, None) == B.FO_ERR_INVALID_ARG
    assert w(desc(), -1, 1, 1, ctypes.byref(size)) == w(desc(), 1, -1, 1, ctypes.byref(size)) == w(desc(), 1, 1, 0, ctypes.byref(size)) == B.FO_ERR_SHAPE
    assert w(desc(), 0, 0, 1, ctypes.byref(size)) == B.FO_OK and size.value >= 64


def test_a_rotary_description_that_does_not_fit_is_refused():
    good = lambda **k: B.fo_rope_desc(k.pop("D", 128), k.pop("q", 8), k.pop("k", 2), k.pop("v", 2), **k)  # noqa: E731
    for rope in (good(D=64), good(q=4), good(k=1), good(v=0), good(R=2), good(dtype="f32")):
        assert append(rope=rope) == B.FO_ERR_INVALID_ARG
    rope = good()
    rope.ready = 0
    assert append(rope=rope) == B.FO_ERR_INVALID_ARG
    rope = good()
    rope.rot_dim = 3
    assert append(rope=rope) == B.FO_ERR_SHAPE
    assert append(rope=good(), q=None) == B.FO_ERR_INVALID_ARG


def test_the_binding_says_what_is_wrong():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="int32 expected"):
        B.fo_paged_batch(torch.zeros(2), torch.zeros(2, 3, **i32), 4)
    with pytest.raises(ValueError, match="sequences, columns"):
        B.fo_paged_batch(torch.zeros(2, **i32), torch.zeros(6, **i32), 4)
    with pytest.raises(ValueError, match="3 values given, 2 expected"):
        B.fo_paged_batch(torch.zeros(3, **i32), torch.zeros(2, 3, **i32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        B.fo_paged_batch(torch.zeros(2, **i32), torch.zeros(2, 3, **i32), 4)
    b, d = batch(), desc()
    q, c = torch.zeros(3, 1024, dtype=torch.bfloat16), torch.zeros(10, 2, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q: 3 rows of 1024"):
        B.fo_paged_attention(d, b, 3, [q[:, :512]], [c], [c], [q], 256, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        B.fo_paged_attention(d, b, 3, [q], [c], [c], [q], 256, stream=0)
    with pytest.raises(ValueError, match="k_cache: 0 tensors|k_cache: .* expected"):
        B.fo_paged_attention(d, b, 3, [256], [c[:5]], [c], [256], 256, stream=0)
    with pytest.raises(ValueError, match="k_cache: torch.bfloat16 given"):
        B.fo_paged_attention(desc(cache_dtype=1), b, 3, [256], [c], [c], [256], 256, stream=0)
    with pytest.raises(ValueError, match="positions"):
        B.fo_kv_append(d, None, b, 3, [256], [256], [256], [256], [256], [256], positions=torch.zeros(3), stream=0)
    with pytest.raises(B.FlashOverlapError) as e:
        B.fo_kv_append(d, None, batch(max_new=0), 3, [256], [256], [256], [256], [256], [256], stream=0)
    assert e.value.code == B.FO_ERR_SHAPE
