"""Thin ctypes binding of libflashoverlap.so (include/flashoverlap.h).

Argument marshalling only: device pointers and streams are taken from torch
tensors / streams, every step of the computation runs in the library's CUDA
kernels. Function names match the C ABI. A non-OK status raises
``FlashOverlapError``. If the library has not been built the first call
raises: there is no CPU or PyTorch fallback.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_int32, c_int64, c_size_t, c_uint64, c_void_p
from typing import List, Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libflashoverlap.so")

FO_OK, FO_ERR_INVALID_ARG, FO_ERR_SHAPE, FO_ERR_DTYPE, FO_ERR_ALIGN = 0, 1, 2, 3, 4
FO_ERR_UNSUPPORTED, FO_ERR_CUDA, FO_ERR_TIMEOUT, FO_ERR_PLAN_INVARIANT = 5, 6, 7, 8
FO_ERR_SCRATCH_LIMIT = 9
FO_NOALLOC_SCRATCH_BYTES = 64 * 1024
OPS = {"ag_gemm": 0, "gemm_rs": 1, "dp_grad_rs": 2, "gemm_ar": 3, "gemm_a2a": 4}
DTYPES = {"bf16": 0, "f32": 1}
SCHEDS = {"rank_adaptive": 0, "sliced": 1}
TRANSPORTS = {"peer_read": 0, "copy": 1}
W_LAYOUTS = {"kn": 0, "nk": 1}
INJECT = {"none": 0, "drop_transfer": 1, "skip_signal": 2, "delay_first_task": 3}
FO_TRACE_STAMPS = 8
FO_TRACE_MAX_CTAS = 1024
TILE_CONFIGS = {"auto": 0, "single": 1}
INTERLEAVES = {"auto": 0, "lockstep": 1, "skewed": 2, "rank_major": 3, "skewed_pairs": 4}
RS_ALGOS = {"direct": 0, "ring": 1}
TAIL_SPLITS = {"auto": 0, "off": 1, "on": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
CACHE_DTYPES = {"bf16": 0, "e4m3": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "wavelength": 2, "parts": 3}
FO_ROPE_MAX_DIM = 256
FO_NORM_MAX_H = 32768
FO_OPS_HEADER = 64                # bytes of a workspace that hold its status
FO_FP8_BLOCK = 128

# Every symbol include/flashoverlap.h declares.
EXPORTED = [
    "fo_plan", "fo_plan_destroy", "fo_plan_table", "fo_plan_transfers", "fo_plan_edges",
    "fo_workspace_size", "fo_workspace_init", "fo_ag_gemm", "fo_gemm_rs", "fo_dp_grad_rs",
    "fo_status_query", "fo_gemm_partials", "fo_reduce_scatter_f32", "fo_all_gather_copy",
    "fo_plan_last_launches", "fo_status_string", "fo_version", "fo_gemm_rs_noalloc", "fo_plan_task_order",
    "fo_gemm_ar", "fo_trace_query", "fo_plan_last_split_tiles", "fo_check_device_pointers",
    "fo_gemm_a2a", "fo_all_to_all_copy", "fo_attn_rs", "fo_attention", "fo_gemm_partials_sharded",
    "fo_rmsnorm", "fo_rmsnorm_bwd", "fo_rmsnorm_bwd_workspace", "fo_quant_fp8", "fo_gemm_fp8",
    "fo_gemm_fp8_workspace", "fo_ops_workspace_init", "fo_ops_status_query", "fo_rope_init", "fo_rope",
    "fo_kv_append", "fo_paged_attention", "fo_paged_attention_workspace",
]


class FlashOverlapError(RuntimeError):
    def __init__(self, code: int, where: str, info=None):
        self.code = code
        self.info = info
        msg = f"{where}: {status_string(code)} (code {code})"
        if info is not None:
            msg += f" info={list(info)}"
        super().__init__(msg)


class PlanDesc(ctypes.Structure):
    _fields_ = [
        ("op", c_int32), ("R", c_int32), ("M", c_int64), ("N", c_int64), ("K", c_int64),
        ("in_dtype", c_int32), ("out_dtype", c_int32), ("sched", c_int32), ("ag_transport", c_int32),
        ("w_layout", c_int32), ("deterministic", c_int32), ("timeout_ns", c_uint64),
        ("fault_inject", c_int32), ("tile_config", c_int32), ("interleave", c_int32), ("rs_algo", c_int32),
        ("trace", c_int32), ("inject_delay_us", c_int32), ("tail_split", c_int32),
        ("reserved", c_int32 * 1),
    ]


class NormDesc(ctypes.Structure):
    _fields_ = [("R", c_int32), ("H", c_int32), ("dtype", c_int32), ("w_dtype", c_int32), ("eps", ctypes.c_float),
                ("w_offset", ctypes.c_float), ("reserved", c_int32 * 2)]


class GemmFp8Desc(ctypes.Structure):
    _fields_ = [("R", c_int32), ("out_dtype", c_int32), ("N", c_int64), ("K", c_int64), ("reserved", c_int32 * 4)]


class RopeDesc(ctypes.Structure):
    _fields_ = [(n, c_int32) for n in ("R", "head_dim", "rot_dim", "heads_q", "heads_k", "heads_v", "layout", "dtype",
                                       "scaling", "reserved")]
    _fields_ += [(n, ctypes.c_double) for n in ("base", "stretch", "trained", "slow", "fast")]
    _fields_ += [("turns", c_uint64 * (FO_ROPE_MAX_DIM // 2)), ("factor", ctypes.c_float), ("ready", c_int32)]


class PagedDesc(ctypes.Structure):
    _fields_ = [(n, c_int32) for n in ("R", "heads_q", "heads_k", "head_dim", "page", "cache_dtype", "window", "sinks")]
    _fields_ += [("scale", ctypes.c_float), ("reserved", c_int32 * 3)]


class PagedBatch(ctypes.Structure):
    _fields_ = [("seqs", c_int32), ("max_new", c_int32), ("pages", c_int64), ("table_cols", c_int64),
                ("lengths", c_void_p), ("starts", c_void_p), ("table", c_void_p)]


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libflashoverlap.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libflashoverlap.so not found at {path}: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    P = c_void_p
    PP = POINTER(c_void_p)
    sig = {
        "fo_plan": ([POINTER(PlanDesc), POINTER(c_void_p)], c_int32),
        "fo_plan_destroy": ([P], None),
        "fo_plan_table": ([P, POINTER(c_int32)], c_int32),
        "fo_plan_task_order": ([P, POINTER(c_int32)], c_int32),
        "fo_plan_transfers": ([P, POINTER(c_int32), c_int32, POINTER(c_int32)], c_int32),
        "fo_plan_edges": ([P, POINTER(c_int32), c_int32, POINTER(c_int32)], c_int32),
        "fo_workspace_size": ([P, POINTER(c_size_t)], c_int32),
        "fo_workspace_init": ([P, P, P], c_int32),
        "fo_ag_gemm": ([P, PP, PP, PP, PP, P, P], c_int32),
        "fo_gemm_rs": ([P, PP, PP, PP, P, P], c_int32),
        "fo_dp_grad_rs": ([P, PP, PP, PP, P, P], c_int32),
        "fo_gemm_rs_noalloc": ([P, PP, PP, PP, P], c_int32),
        "fo_gemm_ar": ([P, PP, PP, PP, P, P], c_int32),
        "fo_gemm_a2a": ([P, PP, PP, PP, P, P], c_int32),
        "fo_all_to_all_copy": ([P, PP, PP, P], c_int32),
        "fo_attn_rs": ([P, PP, PP, PP, PP, PP, PP, c_int32, c_int32, P, P], c_int32),
        "fo_attention": ([P, PP, PP, PP, PP, c_int32, c_int32, P, P], c_int32),
        "fo_gemm_partials_sharded": ([P, PP, PP, PP, P, P], c_int32),
        "fo_status_query": ([P, P, P, POINTER(c_int32)], c_int32),
        "fo_trace_query": ([P, P, P, POINTER(ctypes.c_uint64), c_int32, POINTER(c_int32)], c_int32),
        "fo_gemm_partials": ([P, PP, PP, PP, P, P], c_int32),
        "fo_reduce_scatter_f32": ([P, PP, PP, P], c_int32),
        "fo_all_gather_copy": ([P, PP, PP, P], c_int32),
        "fo_plan_last_launches": ([P], c_int32),
        "fo_plan_last_split_tiles": ([P], c_int32),
        "fo_check_device_pointers": ([c_int32, PP, P], c_int32),
        "fo_rmsnorm": ([POINTER(NormDesc), c_int64, PP, PP, P, PP, PP, PP, PP, PP, P], c_int32),
        "fo_rmsnorm_bwd": ([POINTER(NormDesc), c_int64, PP, PP, PP, P, PP, PP, P, P, P], c_int32),
        "fo_rmsnorm_bwd_workspace": ([POINTER(NormDesc), c_int64, POINTER(c_size_t)], c_int32),
        "fo_quant_fp8": ([c_int32, c_int64, c_int64, c_int32, c_int32, PP, PP, PP, PP, PP, P], c_int32),
        "fo_gemm_fp8": ([POINTER(GemmFp8Desc), c_int64, PP, PP, PP, PP, PP, P, P], c_int32),
        "fo_gemm_fp8_workspace": ([POINTER(GemmFp8Desc), c_int64, POINTER(c_size_t)], c_int32),
        "fo_ops_workspace_init": ([P, c_size_t, P], c_int32),
        "fo_ops_status_query": ([P, P, POINTER(c_int32)], c_int32),
        "fo_rope_init": ([POINTER(RopeDesc)], c_int32),
        "fo_rope": ([POINTER(RopeDesc), c_int64, P, c_int32, PP, PP, PP, POINTER(c_int64), PP, PP, PP,
                     POINTER(c_int64), c_int32, P], c_int32),
        "fo_kv_append": ([POINTER(PagedDesc), POINTER(RopeDesc), POINTER(PagedBatch), c_int64, P, c_int32, PP, PP, PP, PP,
                          POINTER(c_int64), PP, PP, PP, PP, P, P], c_int32),
        "fo_paged_attention": ([POINTER(PagedDesc), POINTER(PagedBatch), c_int64, PP, POINTER(c_int64), PP, PP, PP, PP, PP,
                                PP, P, P], c_int32),
        "fo_paged_attention_workspace": ([POINTER(PagedDesc), c_int32, c_int64, c_int32, POINTER(c_size_t)], c_int32),
        "fo_status_string": ([c_int32], ctypes.c_char_p),
        "fo_version": ([], c_int32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return load().fo_status_string(code).decode()
    except Exception:  # library missing: still give a readable message
        return f"status {code}"


def _check(code: int, where: str):
    if code != FO_OK:
        raise FlashOverlapError(code, where)


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("tensors passed to libflashoverlap must be contiguous")
        if not getattr(x, "is_cuda", True) and not x.is_pinned():
            raise ValueError("tensors passed to libflashoverlap must be CUDA tensors (or pinned host memory)")
        return x.data_ptr()
    raise TypeError(f"cannot take a device pointer from {type(x)!r}")


def _ptr_array(xs: Optional[Sequence]):
    if xs is None:
        return None
    arr = (c_void_p * len(xs))()
    for i, x in enumerate(xs):
        arr[i] = _ptr(x)
    return arr


_current_stream = None


def _stream(s) -> int:
    if s is None:
        global _current_stream
        if _current_stream is None:
            import torch
            if not torch.cuda.is_available():
                return 0
            raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            # The stream's address alone, where torch gives it: a Stream object for every call took 3 us.
            _current_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


class Plan:
    """Owns an fo_plan_t; freed with fo_plan_destroy when collected."""

    def __init__(self, handle: int, desc: PlanDesc):
        self.handle = handle
        self.desc = desc
        self.R = desc.R

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.fo_plan_destroy(self.handle)
            self.handle = None

    @property
    def _as_parameter_(self):
        return c_void_p(self.handle)


def fo_plan(op: str, R: int, M: int, N: int, K: int, *, in_dtype="bf16", out_dtype=None,
            sched="rank_adaptive", ag_transport="peer_read", w_layout="kn", deterministic=False,
            timeout_ns=0, fault_inject="none", tile_config="auto", interleave="auto",
            rs_algo="direct", trace=False, inject_delay_us=0, tail_split="auto") -> Plan:
    lib = load()
    if out_dtype is None:
        out_dtype = "bf16" if op in ("ag_gemm", "gemm_a2a") else "f32"
    d = PlanDesc()
    d.op = OPS[op]
    d.R = R
    d.M, d.N, d.K = M, N, K
    d.in_dtype = DTYPES[in_dtype]
    d.out_dtype = DTYPES[out_dtype]
    d.sched = SCHEDS[sched]
    d.ag_transport = TRANSPORTS[ag_transport]
    d.w_layout = W_LAYOUTS[w_layout]
    d.deterministic = 1 if deterministic else 0
    d.timeout_ns = timeout_ns
    d.fault_inject = INJECT[fault_inject]
    d.tile_config = TILE_CONFIGS[tile_config]
    d.interleave = INTERLEAVES[interleave]
    d.rs_algo = RS_ALGOS[rs_algo]
    d.trace = 1 if trace else 0
    d.inject_delay_us = inject_delay_us
    d.tail_split = TAIL_SPLITS[tail_split]
    h = c_void_p()
    _check(lib.fo_plan(ctypes.byref(d), ctypes.byref(h)), "fo_plan")
    return Plan(h.value, d)


def fo_plan_destroy(plan: Plan) -> None:
    if plan.handle:
        load().fo_plan_destroy(plan.handle)
        plan.handle = None


def fo_plan_table(plan: Plan) -> List[List[int]]:
    R = plan.R
    buf = (c_int32 * (R * R))()
    _check(load().fo_plan_table(plan, buf), "fo_plan_table")
    return [[buf[r * R + s] for s in range(R)] for r in range(R)]


def fo_plan_task_order(plan: Plan):
    """[(rank, step), ...] in the order the kernel runs the chunk tasks."""
    n = plan.R * plan.R
    buf = (c_int32 * (2 * n))()
    _check(load().fo_plan_task_order(plan, buf), "fo_plan_task_order")
    return [(buf[2 * i], buf[2 * i + 1]) for i in range(n)]


def _quads(fn, plan: Plan, what: str):
    n = c_int32()
    fn(plan, None, 0, ctypes.byref(n))
    cap = max(n.value, 1)
    buf = (c_int32 * (4 * cap))()
    _check(fn(plan, buf, cap, ctypes.byref(n)), what)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n.value)]


def fo_plan_transfers(plan: Plan):
    return _quads(load().fo_plan_transfers, plan, "fo_plan_transfers")


def fo_plan_edges(plan: Plan):
    return _quads(load().fo_plan_edges, plan, "fo_plan_edges")


def fo_workspace_size(plan: Plan) -> int:
    n = c_size_t()
    _check(load().fo_workspace_size(plan, ctypes.byref(n)), "fo_workspace_size")
    return n.value


def fo_workspace_init(plan: Plan, ws, stream=None) -> None:
    _check(load().fo_workspace_init(plan, _ptr(ws), _stream(stream)), "fo_workspace_init")


def fo_gemm_rs(plan: Plan, X, W, Y, ws, stream=None) -> None:
    _check(load().fo_gemm_rs(plan, _ptr_array(X), _ptr_array(W), _ptr_array(Y), _ptr(ws), _stream(stream)),
           "fo_gemm_rs")


def fo_gemm_ar(plan: Plan, X, W, Y, ws, stream=None) -> None:
    _check(load().fo_gemm_ar(plan, _ptr_array(X), _ptr_array(W), _ptr_array(Y), _ptr(ws), _stream(stream)),
           "fo_gemm_ar")


def fo_gemm_a2a(plan: Plan, X, W, Y, ws, stream=None) -> None:
    _check(load().fo_gemm_a2a(plan, _ptr_array(X), _ptr_array(W), _ptr_array(Y), _ptr(ws), _stream(stream)),
           "fo_gemm_a2a")


def fo_all_to_all_copy(plan: Plan, P, Y, stream=None) -> None:
    _check(load().fo_all_to_all_copy(plan, _ptr_array(P), _ptr_array(Y), _stream(stream)), "fo_all_to_all_copy")


def fo_attn_rs(plan: Plan, Q, K, V, Wo, O, Y, heads: int, causal: bool, ws, stream=None) -> None:
    _check(load().fo_attn_rs(plan, _ptr_array(Q), _ptr_array(K), _ptr_array(V), _ptr_array(Wo), _ptr_array(O),
                             _ptr_array(Y), int(heads), 1 if causal else 0, _ptr(ws), _stream(stream)),
           "fo_attn_rs")


def fo_attention(plan: Plan, Q, K, V, O, heads: int, causal: bool, ws, stream=None) -> None:
    _check(load().fo_attention(plan, _ptr_array(Q), _ptr_array(K), _ptr_array(V), _ptr_array(O), int(heads),
                               1 if causal else 0, _ptr(ws), _stream(stream)),
           "fo_attention")


def fo_ag_gemm(plan: Plan, X, W, Y, G=None, ws=None, stream=None) -> None:
    _check(load().fo_ag_gemm(plan, _ptr_array(X), _ptr_array(W), _ptr_array(Y), _ptr_array(G), _ptr(ws),
                             _stream(stream)), "fo_ag_gemm")


def fo_gemm_rs_noalloc(plan: Plan, X, W, Y, stream=None) -> None:
    """fo_gemm_rs without a workspace (static device scratch; see the header)."""
    _check(load().fo_gemm_rs_noalloc(plan, _ptr_array(X), _ptr_array(W), _ptr_array(Y), _stream(stream)),
           "fo_gemm_rs_noalloc")


def fo_dp_grad_rs(plan: Plan, X, dY, dW, ws, stream=None) -> None:
    _check(load().fo_dp_grad_rs(plan, _ptr_array(X), _ptr_array(dY), _ptr_array(dW), _ptr(ws),
                                _stream(stream)), "fo_dp_grad_rs")


def fo_gemm_partials(plan: Plan, A, B, P, ws, stream=None) -> None:
    _check(load().fo_gemm_partials(plan, _ptr_array(A), _ptr_array(B), _ptr_array(P), _ptr(ws),
                                   _stream(stream)), "fo_gemm_partials")


def fo_gemm_partials_sharded(plan: Plan, A_shards, B, P, ws, stream=None) -> None:
    _check(load().fo_gemm_partials_sharded(plan, _ptr_array(A_shards), _ptr_array(B), _ptr_array(P), _ptr(ws),
                                           _stream(stream)), "fo_gemm_partials_sharded")


def fo_check_device_pointers(ptrs, stream=None) -> int:
    """Status of fo_check_device_pointers for raw addresses (ints): FO_OK
    when the current device can use every one of them."""
    arr = (c_void_p * len(ptrs))(*[int(p) for p in ptrs])
    return int(load().fo_check_device_pointers(len(ptrs), arr, _stream(stream)))


def fo_reduce_scatter_f32(plan: Plan, P, Y, stream=None) -> None:
    _check(load().fo_reduce_scatter_f32(plan, _ptr_array(P), _ptr_array(Y), _stream(stream)),
           "fo_reduce_scatter_f32")


def fo_all_gather_copy(plan: Plan, X, G, stream=None) -> None:
    _check(load().fo_all_gather_copy(plan, _ptr_array(X), _ptr_array(G), _stream(stream)), "fo_all_gather_copy")


def fo_status_query(plan: Plan, ws, stream=None):
    """Returns (status code, [code, rank, step, chunk]) without raising."""
    info = (c_int32 * 4)()
    code = load().fo_status_query(plan, _ptr(ws), _stream(stream), info)
    return code, list(info)


def fo_trace_query(plan: Plan, ws, stream=None):
    """Per-CTA timestamps of the last traced launch: a list with one row of
    FO_TRACE_STAMPS ints (ns) per CTA."""
    cap = FO_TRACE_MAX_CTAS
    buf = (ctypes.c_uint64 * (cap * FO_TRACE_STAMPS))()
    n = c_int32()
    _check(load().fo_trace_query(plan, _ptr(ws), _stream(stream), buf, cap, ctypes.byref(n)), "fo_trace_query")
    m = min(n.value, cap)
    return [[buf[i * FO_TRACE_STAMPS + j] for j in range(FO_TRACE_STAMPS)] for i in range(m)]


def trace_summary(stamps):
    """Launch span, end of the math and exposed tail (all ns) from
    fo_trace_query's rows: the tail is the time the last transfer was still
    running after the last MMA had completed."""
    start = min(r[0] for r in stamps)
    mma_end = max(r[1] for r in stamps)
    xfer_end = max(max(r[2:6]) for r in stamps)
    end = max(r[6] for r in stamps)
    return {"span_ns": end - start, "mma_end_ns": mma_end - start, "transfers_end_ns": xfer_end - start,
            "exposed_tail_ns": max(0, xfer_end - mma_end)}


# ---- operators between the residual stream and the attention

_marshal = None


class _NoMarshal:
    """In the module's place where it is missing: leaves every call to the code below."""

    @staticmethod
    def _leave(*args):
        return -1

    rmsnorm = rmsnorm_bwd = quant_fp8 = gemm_fp8 = rope = kv_append = paged_attention = _leave


def _native():
    """The marshalling module (csrc/fo_marshal.cpp): makes a call whose arguments are right and returns its status, or
    returns -1 and leaves it to the code below, which says what is wrong. Where it was not built for this torch and
    interpreter, the code below does all of the work (a decode step's norm takes 15.4 us of host time then, 4.9 with it)."""
    global _marshal
    if _marshal is None:
        import importlib.machinery
        import importlib.util
        load()
        try:
            import torch  # noqa: F401  (whose libraries the module is linked to)
            from .build import marshal_path
            path = marshal_path()
            loader = importlib.machinery.ExtensionFileLoader("_fo_marshal", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_fo_marshal", path, loader=loader))
            loader.exec_module(module)
        except (ImportError, OSError) as e:
            import warnings
            warnings.warn(f"the operators' arguments are checked in Python, for want of the native module: {e}", RuntimeWarning)
            module = _NoMarshal
        _marshal = module
    return _marshal


_TORCH_DTYPES = None


def _types():
    """DTYPES code -> the torch types that may stand for it (8-bit values: e4m3 or raw bytes; without torch, addresses alone)."""
    global _TORCH_DTYPES
    if _TORCH_DTYPES is None:
        try:
            import torch
        except ImportError:
            return {0: (), 1: (), "q": ()}
        _TORCH_DTYPES = {0: (torch.bfloat16,), 1: (torch.float32,), "q": (torch.float8_e4m3fn, torch.uint8)}
    return _TORCH_DTYPES


def _refuse(x, n: int, types, what: str):
    """Raise for what _address found wrong (all but the host memory that can be used after all)."""
    if x.dtype not in types:
        raise ValueError(f"{what}: {x.dtype} given, {' or '.join(map(str, types))} expected")
    if x.numel() != n:
        raise ValueError(f"{what}: {x.numel()} values given, {n} expected")
    _ptr(x)


def _address(x, n: int, types, what: str) -> int:
    """The address of x: a dense CUDA tensor of n values of one of `types`, or a raw address."""
    if type(x) is int:
        return x
    if x is None:
        raise ValueError(f"{what}: None given, a tensor or an address expected")
    if x.dtype not in types or x.numel() != n or not x.is_contiguous() or not x.is_cuda:
        _refuse(x, n, types, what)
    return x.data_ptr()


# These calls are made once a layer on a few rows in serving, so their marshalling counts: about 0.5 us a tensor.
_ARRAYS = [None] + [c_void_p * n for n in range(1, 17)]


def _array_of(R: int):
    return _ARRAYS[R] if 0 < R <= 16 else c_void_p * max(R, 0)


def _addresses(xs, R: int, n: int, types, what: str):
    if xs is None:
        return None
    if len(xs) != R:
        raise ValueError(f"{what}: {len(xs)} tensors given, one for each of {R} ranks expected")
    at, last = [], None
    for x in xs:
        if x is not last or x is None:
            here, last = _address(x, n, types, what), x
        at.append(here)
    return _array_of(R)(*at)


def fo_norm_desc(H: int, *, R: int = 1, dtype="bf16", w_dtype=None, eps: float = 1e-6, w_offset: float = 0.0) -> NormDesc:
    """Description of an RMSNorm of H columns over R shards of rows (the weight has the rows' dtype unless w_dtype
    says otherwise)."""
    d = NormDesc()
    d.R, d.H, d.eps, d.w_offset = R, H, eps, w_offset
    d.dtype, d.w_dtype = DTYPES[dtype], DTYPES[dtype if w_dtype is None else w_dtype]
    return d


def fo_rmsnorm(desc: NormDesc, rows: int, x, residual, weight, h=None, y=None, q=None, scale=None, rstd=None,
               stream=None) -> None:
    """x, residual, h, y [rows, H], q [rows, H] in 8 bits, scale [rows, ceil(H/128)], rstd [rows]: one tensor for each
    shard; all but x and weight may be None (see the header for what is computed)."""
    code = (_marshal or _native()).rmsnorm(desc, rows, x, residual, weight, h, y, q, scale, rstd, stream)
    if code == FO_OK:
        return
    if code > 0:
        _check(code, "fo_rmsnorm")
    R, H, t = desc.R, desc.H, _types()
    n, types = rows * H, t[desc.dtype]
    groups = rows * -(-H // FO_FP8_BLOCK)
    _check(load().fo_rmsnorm(desc, rows, _addresses(x, R, n, types, "x"),
                             _addresses(residual, R, n, types, "residual"),
                             _address(weight, H, t[desc.w_dtype], "weight"), _addresses(h, R, n, types, "h"),
                             _addresses(y, R, n, types, "y"), _addresses(q, R, n, t["q"], "q"),
                             _addresses(scale, R, groups, t[1], "scale"),
                             _addresses(rstd, R, rows, t[1], "rstd"), _stream(stream)), "fo_rmsnorm")


def fo_rmsnorm_bwd_workspace(desc: NormDesc, rows: int) -> int:
    n = c_size_t()
    _check(load().fo_rmsnorm_bwd_workspace(desc, rows, ctypes.byref(n)), "fo_rmsnorm_bwd_workspace")
    return n.value


def fo_rmsnorm_bwd(desc: NormDesc, rows: int, dy, dh, h, weight, rstd, dx, dweight=None, ws=None, stream=None) -> None:
    """dy, dh (may be None), h, dx [rows, H] and rstd [rows]: one tensor for each shard; dweight [H] fp32 or None."""
    code = (_marshal or _native()).rmsnorm_bwd(desc, rows, dy, dh, h, weight, rstd, dx, dweight, ws, stream)
    if code == FO_OK:
        return
    if code > 0:
        _check(code, "fo_rmsnorm_bwd")
    R, H, t = desc.R, desc.H, _types()
    n, types = rows * H, t[desc.dtype]
    if ws is not None and not isinstance(ws, int) and ws.numel() * ws.element_size() < fo_rmsnorm_bwd_workspace(desc, rows):
        raise ValueError("fo_rmsnorm_bwd: the workspace is smaller than fo_rmsnorm_bwd_workspace says")
    _check(load().fo_rmsnorm_bwd(desc, rows, _addresses(dy, R, n, types, "dy"),
                                 _addresses(dh, R, n, types, "dh"), _addresses(h, R, n, types, "h"),
                                 _address(weight, H, t[desc.w_dtype], "weight"),
                                 _addresses(rstd, R, rows, t[1], "rstd"), _addresses(dx, R, n, types, "dx"),
                                 None if dweight is None else _address(dweight, H, t[1], "dweight"), _ptr(ws),
                                 _stream(stream)), "fo_rmsnorm_bwd")


def fo_quant_fp8(rows: int, cols: int, x, q, scale, qt=None, scale_t=None, *, block_rows: int = 1, dtype=None,
                 stream=None) -> None:
    """x [rows, cols] -> q in 8 bits and scale (one tensor for each rank); block_rows 1: scales of 1 x 128 values,
    128: of 128 x 128, with the transposed copy qt [cols, rows] and scale_t if given. The dtype is x's own unless
    x holds raw addresses."""
    t = _types()
    if dtype is None:
        if not len(x) or x[0] is None or isinstance(x[0], int):
            raise ValueError("x: tensors expected, or addresses and their dtype")
        dtype = "bf16" if x[0].dtype in t[0] else "f32"
    R, code = len(x), DTYPES[dtype]
    status = (_marshal or _native()).quant_fp8(rows, cols, code, block_rows, x, q, scale, qt, scale_t, stream)
    if status == FO_OK:
        return
    if status > 0:
        _check(status, "fo_quant_fp8")
    up, across = (-(-rows // block_rows) if block_rows > 0 else 0), -(-cols // FO_FP8_BLOCK)
    _check(load().fo_quant_fp8(R, rows, cols, code, block_rows, _addresses(x, R, rows * cols, t[code], "x"),
                               _addresses(q, R, rows * cols, t["q"], "q"),
                               _addresses(scale, R, up * across, t[1], "scale"),
                               _addresses(qt, R, rows * cols, t["q"], "qt"),
                               _addresses(scale_t, R, up * across, t[1], "scale_t"), _stream(stream)),
           "fo_quant_fp8")


def fo_gemm_fp8_desc(N: int, K: int, *, R: int = 1, out_dtype="bf16") -> GemmFp8Desc:
    d = GemmFp8Desc()
    d.R, d.N, d.K, d.out_dtype = R, N, K, DTYPES[out_dtype]
    return d


def fo_gemm_fp8_workspace(desc: GemmFp8Desc, M: int) -> int:
    n = c_size_t()
    _check(load().fo_gemm_fp8_workspace(desc, M, ctypes.byref(n)), "fo_gemm_fp8_workspace")
    return n.value


def fo_gemm_fp8(desc: GemmFp8Desc, M: int, A, sA, W, sW, Y, ws, stream=None) -> None:
    """Y_r [M, N] = (A_r scaled by sA_r) (W_r scaled by sW_r)^T: A [M, K] and W [N, K] in 8 bits, sA [M, ceil(K/128)],
    sW [ceil(N/128), ceil(K/128)]; one tensor for each rank."""
    code = (_marshal or _native()).gemm_fp8(desc, M, A, sA, W, sW, Y, ws, stream)
    if code == FO_OK:
        return
    if code > 0:
        _check(code, "fo_gemm_fp8")
    R, N, K, t = desc.R, desc.N, desc.K, _types()
    k = -(-K // FO_FP8_BLOCK)
    if not isinstance(ws, int) and ws.numel() * ws.element_size() < fo_gemm_fp8_workspace(desc, M):
        raise ValueError("fo_gemm_fp8: the workspace is smaller than fo_gemm_fp8_workspace says")
    _check(load().fo_gemm_fp8(desc, M, _addresses(A, R, M * K, t["q"], "A"),
                              _addresses(sA, R, M * k, t[1], "sA"), _addresses(W, R, N * K, t["q"], "W"),
                              _addresses(sW, R, -(-N // FO_FP8_BLOCK) * k, t[1], "sW"),
                              _addresses(Y, R, M * N, t[desc.out_dtype], "Y"), _ptr(ws), _stream(stream)),
           "fo_gemm_fp8")


def fo_ops_workspace_init(ws, stream=None) -> None:
    """Zero a workspace (a tensor) before its first use."""
    _check(load().fo_ops_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "fo_ops_workspace_init")


def fo_ops_status_query(ws, stream=None):
    """Returns (status code, info) without raising, like fo_status_query."""
    info = (c_int32 * 4)()
    code = load().fo_ops_status_query(_ptr(ws), _stream(stream), info)
    return code, list(info)


def fo_rope_desc(head_dim: int, heads_q: int, heads_k: int = 0, heads_v: int = 0, *, R: int = 1, rot_dim=None,
                 layout="half", dtype="bf16", base: float = 10000.0, scaling="none", stretch: float = 1.0,
                 trained: float = 0.0, slow: float = 0.0, fast: float = 0.0) -> RopeDesc:
    """Description of the rotary positions of heads_q + heads_k heads a rank, heads_v more copied (fo_rope_init
    checks it and fills in the pairs' frequencies)."""
    d = RopeDesc()
    d.R, d.head_dim, d.rot_dim = R, head_dim, head_dim if rot_dim is None else rot_dim
    d.heads_q, d.heads_k, d.heads_v = heads_q, heads_k, heads_v
    d.layout, d.dtype, d.scaling = ROPE_LAYOUTS[layout], DTYPES[dtype], ROPE_SCALINGS[scaling]
    d.base, d.stretch, d.trained, d.slow, d.fast = base, stretch, trained, slow, fast
    _check(load().fo_rope_init(d), "fo_rope_init")
    return d


def _rows_of(xs, R: int, rows: int, width: int, types, what: str):
    """Addresses and the common row stride of R matrices [rows, width] whose rows are dense (parts of packed rows
    among them)."""
    if xs is None or len(xs) != R:
        raise ValueError(f"{what}: {0 if xs is None else len(xs)} tensors given, one for each of {R} ranks expected")
    ld, at, shape = None, [], (rows, width)
    for x in xs:
        if type(x) is int:
            at.append(x)
            continue
        if x is None:
            raise ValueError(f"{what}: None given, a tensor or an address expected")
        if x.dtype not in types:
            raise ValueError(f"{what}: {x.dtype} given, {' or '.join(map(str, types))} expected")
        if x.shape != shape:
            raise ValueError(f"{what}: {rows} rows of {width} dense values expected, {tuple(x.shape)} given")
        up, across = x.stride()
        if across != 1 and width > 1 and rows > 0:
            raise ValueError(f"{what}: {rows} rows of {width} dense values expected, strides {up} and {across} given")
        if rows <= 1:
            up = width
        if up != ld:
            if ld is not None:
                raise ValueError(f"{what}: every rank's rows need the same stride")
            ld = up
        if not x.is_cuda and not x.is_pinned():
            raise ValueError("tensors passed to libflashoverlap must be CUDA tensors (or pinned host memory)")
        at.append(x.data_ptr())
    return _array_of(R)(*at), width if ld is None else ld


def _positions(positions, rows: int):
    """Address and bytes of `rows` positions: an int32 or int64 tensor, a raw address (of int64), or None."""
    if positions is None:
        return 0, 8
    if isinstance(positions, int):
        return positions, 8
    size = positions.element_size()
    if positions.is_floating_point() or size not in (4, 8):
        raise ValueError(f"positions: int32 or int64 expected, {positions.dtype} given")
    return _address(positions, rows, (positions.dtype,), "positions"), size


def fo_rope(desc: RopeDesc, rows: int, positions, q_in, k_in, v_in, q_out, k_out, v_out, *, inverse: bool = False,
            stream=None) -> None:
    """Turn Q and K by their positions ([rows] int32 or int64, None: 0, 1, ...) and copy V; one matrix [rows, heads *
    head_dim] for each rank, whose rows may be parts of packed ones; k_*, v_* are not looked at without heads of
    their kind. inverse: turn back (the gradient)."""
    code = (_marshal or _native()).rope(desc, rows, positions, q_in, k_in, v_in, q_out, k_out, v_out, inverse, stream)
    if code == FO_OK:
        return
    if code > 0:
        _check(code, "fo_rope")
    types = _types()[desc.dtype]
    D, R = desc.head_dim, desc.R
    ins, outs, ld_in, ld_out = [], [], (c_int64 * 3)(), (c_int64 * 3)()
    for j, (heads, i, o, what) in enumerate(((desc.heads_q, q_in, q_out, "Q"), (desc.heads_k, k_in, k_out, "K"),
                                             (desc.heads_v, v_in, v_out, "V"))):
        if heads == 0:
            ins.append(None)
            outs.append(None)
            continue
        a, ld_in[j] = _rows_of(i, R, rows, heads * D, types, what)
        b, ld_out[j] = _rows_of(o, R, rows, heads * D, types, what)
        ins.append(a)
        outs.append(b)
    at, size = _positions(positions, rows)
    _check(load().fo_rope(desc, rows, at, size, *ins, ld_in, *outs, ld_out, 1 if inverse else 0, _stream(stream)),
           "fo_rope")


# ---- serving from a paged cache of keys and values

def fo_paged_desc(heads_q: int, heads_k: int, *, head_dim: int = 128, R: int = 1, page: int = 64, cache="bf16",
                  window: int = 0, sinks: int = 0, scale: float = 0.0) -> PagedDesc:
    """Description of a paged cache and of the attention over it: heads a rank, tokens a page, how the cache is kept
    ("bf16" or "e4m3" with a scale for each token's head), how many tokens a query sees (0: all before it), the first
    tokens that stay visible, the scores' scale (0: 1 / sqrt(head_dim))."""
    d = PagedDesc()
    d.R, d.heads_q, d.heads_k, d.head_dim, d.page = R, heads_q, heads_k, head_dim, page
    d.cache_dtype, d.window, d.sinks, d.scale = CACHE_DTYPES[cache], window, sinks, scale
    return d


def _whole(x, n: Optional[int], what: str) -> int:
    """The address of x, a dense int32 CUDA tensor of n values (None: any number), or a raw address."""
    if type(x) is int:
        return x
    if str(x.dtype) != "torch.int32":
        raise ValueError(f"{what}: int32 expected, {x.dtype} given")
    return _address(x, x.numel() if n is None else n, (x.dtype,), what)


def fo_paged_batch(lengths, table, pages: int, *, starts=None, max_new: int = 1) -> PagedBatch:
    """The sequences of a call: lengths [seqs] with the new tokens, table [seqs, columns] of page numbers, starts
    [seqs + 1] of the new tokens' rows (None: one new token a sequence, sequence b's in row b), int32; pages of each
    rank's cache; the most new tokens of a sequence. The tensors are kept, and what they hold is read when a call runs."""
    b = PagedBatch()
    if table.dim() != 2:
        raise ValueError(f"table: [sequences, columns] expected, {tuple(table.shape)} given")
    b.seqs, b.table_cols = table.shape
    b.max_new, b.pages = max_new, pages
    b.lengths, b.table = _whole(lengths, b.seqs, "lengths"), _whole(table, None, "table")
    b.starts = None if starts is None else _whole(starts, b.seqs + 1, "starts")
    b.kept = (lengths, table, starts)
    return b


def _cache_of(desc: PagedDesc, batch: PagedBatch):
    """Values of a rank's cache, its scales, and the types of the cache."""
    slots = batch.pages * desc.heads_k * desc.page
    return slots * desc.head_dim, slots, _types()["q" if desc.cache_dtype == 1 else 0]


def fo_kv_append(desc: PagedDesc, rope: Optional[RopeDesc], batch: PagedBatch, rows: int, q, k, v, q_out, k_cache, v_cache,
                 k_scale=None, v_scale=None, positions=None, ws=None, stream=None) -> None:
    """Append the batch's new tokens to each rank's cache, turned by `rope` (None: as they are) at their positions in
    their sequences (or at positions [rows], int32 or int64), and turn their queries. q, q_out [rows, heads_q *
    head_dim], k, v [rows, heads_k * head_dim]: one matrix for each rank, whose rows may be parts of packed ones;
    k_cache, v_cache [pages, heads_k, page, head_dim], k_scale, v_scale [pages, heads_k, page] (8 bits only); ws: a
    workspace that takes the status of what the device finds wrong, or None."""
    code = (_marshal or _native()).kv_append(desc, rope, batch, rows, q, k, v, q_out, k_cache, v_cache, k_scale, v_scale,
                                             positions, ws, stream)
    if code == FO_OK:
        return
    if code > 0:
        _check(code, "fo_kv_append")
    R, D, types = desc.R, desc.head_dim, _types()
    values, slots, kept = _cache_of(desc, batch)
    ld, rows_of = (c_int64 * 4)(), []
    for j, (x, heads, what) in enumerate(((q, desc.heads_q, "q"), (k, desc.heads_k, "k"), (v, desc.heads_k, "v"),
                                          (q_out, desc.heads_q, "q_out"))):
        a, ld[j] = _rows_of(x, R, rows, heads * D, types[0], what)
        rows_of.append(a)
    at, size = _positions(positions, rows)
    if ws is not None and not isinstance(ws, int) and ws.numel() * ws.element_size() < FO_OPS_HEADER:
        raise ValueError(f"fo_kv_append: the workspace is smaller than its status, {FO_OPS_HEADER} bytes")
    _check(load().fo_kv_append(desc, rope, batch, rows, at, size, *rows_of, ld,
                               _addresses(k_cache, R, values, kept, "k_cache"), _addresses(v_cache, R, values, kept, "v_cache"),
                               _addresses(k_scale, R, slots, types[1], "k_scale"),
                               _addresses(v_scale, R, slots, types[1], "v_scale"), _ptr(ws), _stream(stream)), "fo_kv_append")


def fo_paged_attention_workspace(desc: PagedDesc, seqs: int, rows: int, max_new: int = 1) -> int:
    n = c_size_t()
    _check(load().fo_paged_attention_workspace(desc, seqs, rows, max_new, ctypes.byref(n)), "fo_paged_attention_workspace")
    return n.value


def fo_paged_attention(desc: PagedDesc, batch: PagedBatch, rows: int, q, k_cache, v_cache, o, ws, k_scale=None, v_scale=None,
                       lse=None, stream=None) -> None:
    """Attention of the batch's new tokens over each rank's cache, which holds them already: q, o [rows, heads_q *
    head_dim] (rows may be parts of wider ones), lse [rows, heads_q] fp32 or None; the cache as in fo_kv_append."""
    code = (_marshal or _native()).paged_attention(desc, batch, rows, q, k_cache, v_cache, o, ws, k_scale, v_scale, lse, stream)
    if code == FO_OK:
        return
    if code > 0:
        _check(code, "fo_paged_attention")
    R, types = desc.R, _types()
    values, slots, kept = _cache_of(desc, batch)
    ld = (c_int64 * 2)()
    q_at, ld[0] = _rows_of(q, R, rows, desc.heads_q * desc.head_dim, types[0], "q")
    o_at, ld[1] = _rows_of(o, R, rows, desc.heads_q * desc.head_dim, types[0], "o")
    if ws is not None and not isinstance(ws, int) and \
            ws.numel() * ws.element_size() < fo_paged_attention_workspace(desc, batch.seqs, rows, batch.max_new):
        raise ValueError("fo_paged_attention: the workspace is smaller than fo_paged_attention_workspace says")
    _check(load().fo_paged_attention(desc, batch, rows, q_at, ld, _addresses(k_cache, R, values, kept, "k_cache"),
                                     _addresses(v_cache, R, values, kept, "v_cache"),
                                     _addresses(k_scale, R, slots, types[1], "k_scale"),
                                     _addresses(v_scale, R, slots, types[1], "v_scale"), o_at,
                                     _addresses(lse, R, rows * desc.heads_q, types[1], "lse"), _ptr(ws), _stream(stream)),
           "fo_paged_attention")


def fo_plan_last_launches(plan: Plan) -> int:
    return load().fo_plan_last_launches(plan)


def fo_plan_last_split_tiles(plan: Plan) -> int:
    return load().fo_plan_last_split_tiles(plan)


def fo_version() -> int:
    return load().fo_version()
