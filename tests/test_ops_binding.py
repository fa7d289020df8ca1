"""The operators' Python calls with and without the native marshalling module, which is there to make them shorter and
may be missing."""
import ctypes
import os
import sysconfig

import pytest
import torch

from ag_gemm_gb300 import binding as B
from ag_gemm_gb300 import build as build_module


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_marshal", None)
    monkeypatch.setattr(build_module, "marshal_path", lambda: str(tmp_path / "none.so"), raising=False)


def test_the_library_is_built_without_the_module(no_module, monkeypatch, capsys):
    def refuse(*args):
        raise RuntimeError("no C++ compiler found")

    monkeypatch.setattr(build_module, "_compile_marshal", refuse)
    before = os.path.getmtime(build_module.LIB)
    assert build_module.build() == build_module.LIB
    assert os.path.getmtime(build_module.LIB) == before      # and not built again for its sake
    assert "no C++ compiler found" in capsys.readouterr().err


def test_the_module_is_of_one_torch_and_one_interpreter(monkeypatch):
    name = os.path.basename(build_module.marshal_path())
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name
    assert os.path.exists(build_module.marshal_path())
    monkeypatch.setattr(build_module, "torch_version", lambda: "0.0.0")
    assert not os.path.exists(build_module.marshal_path())   # what another torch's build left is not taken


def test_calls_without_the_module_refuse_what_they_refuse_with_it(no_module):
    with pytest.warns(RuntimeWarning, match="native module"):
        with pytest.raises(B.FlashOverlapError) as e:
            B.fo_rmsnorm(B.fo_norm_desc(256), -1, [256], None, 256, [256], stream=0)
    assert e.value.code == B.FO_ERR_SHAPE
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.fo_rmsnorm(B.fo_norm_desc(256), 4, [x], None, x[0], [x], stream=0)
    with pytest.raises(ValueError, match="expected"):
        B.fo_quant_fp8(5, 256, [x], [x], [x], stream=0)
    B.fo_quant_fp8(0, 128, [256], [256], [256], dtype="f32", stream=0)
    for call in (lambda: B.fo_rmsnorm_bwd(B.fo_norm_desc(256), -1, [256], None, [256], 256, [256], [256], stream=0),
                 lambda: B.fo_gemm_fp8(B.fo_gemm_fp8_desc(64, 128), -1, [256], [256], [256], [256], [256], 256, stream=0),
                 lambda: B.fo_rope(B.fo_rope_desc(128, 2), -1, None, [256], None, None, [256], None, None, stream=0)):
        with pytest.raises(B.FlashOverlapError) as e:
            call()
        assert e.value.code == B.FO_ERR_SHAPE


def test_calls_refuse_missing_tensors():
    d, x = B.fo_norm_desc(256), torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: None given"):
        B.fo_rmsnorm(d, 4, [None], None, 256, [256], stream=0)
    with pytest.raises(ValueError, match="q: None given"):
        B.fo_quant_fp8(4, 256, [256], [None], [256], dtype="bf16", stream=0)
    for bad in ([], [None], [256]):
        with pytest.raises(ValueError, match="dtype"):
            B.fo_quant_fp8(4, 256, bad, [256], [256], stream=0)
    r = B.fo_rope_desc(128, 2, 1)
    for k in (None, [None], []):
        with pytest.raises(ValueError, match="K: "):
            B.fo_rope(r, 4, None, [256], k, None, [256], [256], None, stream=0)
    with pytest.raises(ValueError, match="weight"):
        B.fo_rmsnorm(d, 4, [256], None, None, [256], stream=0)


@pytest.mark.parametrize("change,code", [
    (dict(heads_q=0, heads_k=0, heads_v=0), B.FO_ERR_SHAPE), (dict(heads_q=0), B.FO_ERR_SHAPE), (dict(heads_k=-1), B.FO_ERR_SHAPE),
    (dict(heads_v=1 << 20), B.FO_ERR_SHAPE), (dict(rot_dim=63), B.FO_ERR_SHAPE), (dict(rot_dim=256), B.FO_ERR_SHAPE),
    (dict(head_dim=0), B.FO_ERR_SHAPE), (dict(R=17), B.FO_ERR_INVALID_ARG), (dict(dtype=7), B.FO_ERR_DTYPE),
    (dict(layout=2), B.FO_ERR_INVALID_ARG), (dict(scaling=-1), B.FO_ERR_INVALID_ARG), (dict(base=0.5), B.FO_ERR_INVALID_ARG),
    (dict(reserved=1), B.FO_ERR_INVALID_ARG)])
def test_rope_refuses_a_description_that_was_spoilt_after_its_check(change, code):
    d = B.fo_rope_desc(128, 2, 1, 1)
    for k, v in change.items():
        setattr(d, k, v)
    one = (ctypes.c_void_p * 17)(*[256] * 17)
    ld = (ctypes.c_int64 * 3)(1 << 40, 1 << 40, 1 << 40)
    assert B.load().fo_rope(d, 4, 256, 8, one, one, one, ld, one, one, one, ld, 0, None) == code


@pytest.mark.gpu
def test_calls_without_the_module_give_the_same(no_module, monkeypatch):
    rows, H, e4m3 = 6, 640, torch.float8_e4m3fn
    g = torch.Generator().manual_seed(1)
    x, res = (torch.randn(rows, H, generator=g).bfloat16().cuda() for _ in range(2))
    w, pos = torch.rand(H, generator=g).bfloat16().cuda(), torch.arange(rows, device="cuda")
    new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731

    def chain():
        d = B.fo_norm_desc(H)
        h, q, s, r = new(rows, H, dtype=torch.bfloat16), new(rows, H, dtype=e4m3), new(rows, 5), new(rows)
        B.fo_rmsnorm(d, rows, [x], [res], w, [h], None, [q], [s], [r])
        dx, dw = torch.zeros_like(x), new(H)
        B.fo_rmsnorm_bwd(d, rows, [x], [res], [h], w, [r], [dx], dw, new(B.fo_rmsnorm_bwd_workspace(d, rows), dtype=torch.uint8))
        wq, ws, y, p = new(rows, H, dtype=e4m3), new(1, 5), new(rows, rows), B.fo_gemm_fp8_desc(rows, H, out_dtype="f32")
        B.fo_quant_fp8(rows, H, [x], [wq], [ws], block_rows=128)
        B.fo_gemm_fp8(p, rows, [q], [s], [wq], [ws], [y], new(B.fo_gemm_fp8_workspace(p, rows), dtype=torch.uint8))
        turned = torch.zeros_like(x)
        B.fo_rope(B.fo_rope_desc(128, 3, 2), rows, pos, [x[:, :384]], [x[:, 384:]], None, [turned[:, :384]], [turned[:, 384:]], None)
        return [h, q.view(torch.uint8), s, r, dx, dw, wq.view(torch.uint8), ws, y, turned]

    with pytest.warns(RuntimeWarning, match="native module"):
        without = chain()
    monkeypatch.undo()
    assert B._marshal is not B._NoMarshal
    assert all(torch.equal(a, b) and torch.count_nonzero(a) for a, b in zip(without, chain()))
