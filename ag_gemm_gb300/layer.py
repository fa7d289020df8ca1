"""The projection GEMMs of one tensor- and sequence-parallel (TP-SP)
transformer layer, forward and backward, on the fused collectives.

The pages name this use: the method is instantiated for the row- and
column-parallel projections of MLP and QKV layers (gist.science, "Technical
Summary" section 2, "Architectural Versatility"), in training forward and
backward (section 3). With R virtual ranks, a sequence of T tokens split
T/R per rank, hidden size H and FFN size F:

forward
    QKV     column-parallel: AG-GEMM      Y_qkv_r = AllGather(x) . Wqkv_r    [H x 3H/R]
    o       row-parallel:    GEMM-RS      h       = RS(attn_r . Wo_r)        [H/R x H]
    up|gate column-parallel: AG-GEMM      Y_ug_r  = AllGather(h) . Wug_r     [H x 2F/R]
    down    row-parallel:    GEMM-RS      y       = RS(act_r . Wd_r)         [F/R x H]
backward (the usual TP-SP duals; the pages do not spell them out)
    row-parallel GEMM-RS Y = RS(X_r . W_r):
        dX_r = AllGather(dY) . W_r^T          AG-GEMM, W read as [N x K]
        dW_r = X_r^T . AllGather(dY)          per-rank weight GEMM (partials)
    column-parallel AG-GEMM Y_r = AllGather(X) . W_r:
        dX   = RS(dY_r . W_r^T)               GEMM-RS, W read as [N x K]
        dW_r = AllGather(X)^T . dY_r          per-rank weight GEMM (partials)
The weight gradients of the row-parallel projections (o, down) are produced
transposed, as AllGather(dY)^T . X_r, i.e. in the nn.Linear layout
[out x in] = [H x H/R] and [H x F/R]: the per-rank GEMM then splits H rows
into R chunks of H/R rows instead of H/R or F/R rows into R chunks (64 or
224 rows for the default shape, which fill 128- and 256-row tiles poorly).
Each weight gradient contracts over all T tokens of an all-gathered
operand; it reads the R token shards where they lie, so no gathered copy
of x, h, dy or dh is written. Those shards are allocated back to back in
rank order, which the weight-gradient call reads as one tensor.

The attention core, the SwiGLU and the norms are not part of the path: their
outputs (attn_r, act_r) and upstream gradients are fixed synthetic tensors.
Every GEMM runs in the library's kernels; this module only allocates
buffers and issues the calls: 12 launches per forward + backward (4
forward collective GEMMs, 4 backward data-gradient collective GEMMs and 4
per-rank weight-gradient GEMMs).
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import Dict, List

import torch

from . import binding as B


@dataclass(frozen=True)
class LayerShape:
    R: int = 8
    T: int = 8192
    H: int = 4096
    F: int = 14336

    def flops(self) -> Dict[str, float]:
        T, H, F = self.T, self.H, self.F
        fwd = 2.0 * T * H * (3 * H) + 2.0 * T * H * H + 2.0 * T * H * (2 * F) + 2.0 * T * F * H
        return {"forward": fwd, "backward": 2 * fwd, "total": 3 * fwd}


def _draw(g, shape, std, device):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(device)


def _ints(g, shape, device):
    return torch.randint(-4, 5, shape, generator=g, dtype=torch.int32).to(torch.bfloat16).to(device)


class TpspLayerProjections:
    """Buffers, plans and launches for one layer's projections (R virtual ranks
    on one GPU). `mode="randn"` draws weights ~N(0, 0.02) and activations /
    gradients ~N(0, 1); `mode="int"` draws integers in [-4, 4] so every sum
    is exact in fp32.

    The weight gradients after an all-gather GEMM (dWqkv, dWug, dWd, dWo)
    contract over the gathered tokens. By default they read the R row shards
    where they lie (fo_gemm_partials_sharded) and the all-gather GEMMs keep
    no gathered copy; `keep_gathered=True` has the all-gather GEMMs write the
    gathered inputs (Gx, Gh, G_dy, G_dh) and the weight gradients read those,
    as a framework that saves the gathered activation for its backward
    would."""

    def __init__(self, shape: LayerShape = LayerShape(), *, device="cuda", seed=4, mode="randn",
                 keep_gathered=False):
        self.s = s = shape
        R, T, H, F = s.R, s.T, s.H, s.F
        if T % R or H % R or F % R:
            raise ValueError("T, H and F must be divisible by R")
        dev = torch.device(device)
        g = torch.Generator().manual_seed(seed)
        w = (lambda shp: _ints(g, shp, dev)) if mode == "int" else (lambda shp: _draw(g, shp, 0.02, dev))
        a = (lambda shp: _ints(g, shp, dev)) if mode == "int" else (lambda shp: _draw(g, shp, 1.0, dev))
        bf, f32 = torch.bfloat16, torch.float32

        def per_rank(shp, dtype=bf):
            return [torch.empty(shp, dtype=dtype, device=dev) for _ in range(R)]

        def token_shards(draw, shp):
            # The R token shards of a sequence-parallel tensor, back to back
            # in rank order: their all-gather is the whole buffer.
            whole = torch.cat([draw(shp) for _ in range(R)]) if draw else torch.empty((R * shp[0], shp[1]),
                                                                                      dtype=bf, device=dev)
            return list(whole.split(shp[0]))

        # weights (each rank's slice)
        self.Wqkv = [w((H, 3 * H // R)) for _ in range(R)]
        self.Wo = [w((H // R, H)) for _ in range(R)]
        self.Wug = [w((H, 2 * F // R)) for _ in range(R)]
        self.Wd = [w((F // R, H)) for _ in range(R)]
        # forward inputs and the synthetic outputs of the skipped parts
        self.x = token_shards(a, (T // R, H))
        self.attn = [a((T, H // R)) for _ in range(R)]
        self.act = [a((T, F // R)) for _ in range(R)]
        # upstream gradients
        self.dy = token_shards(a, (T // R, H))              # into the down projection's output
        self.dh = token_shards(a, (T // R, H))              # into the o projection's output
        self.dug = [a((T, 2 * F // R)) for _ in range(R)]   # into up|gate's output (through SwiGLU)
        self.dqkv = [a((T, 3 * H // R)) for _ in range(R)]  # into QKV's output (through attention)
        # forward outputs (and, if kept, the gathered inputs for the weight gradients)
        self.keep_gathered = keep_gathered
        gathered = per_rank if keep_gathered else (lambda shp: None)
        self.Gx, self.Gh = gathered((T, H)), gathered((T, H))
        self.y_qkv, self.y_ug = per_rank((T, 3 * H // R)), per_rank((T, 2 * F // R))
        self.h, self.y = token_shards(None, (T // R, H)), per_rank((T // R, H))
        # backward outputs
        self.G_dy, self.G_dh = gathered((T, H)), gathered((T, H))
        self.d_act, self.d_attn = per_rank((T, F // R)), per_rank((T, H // R))
        self.d_h_from_ug, self.d_x = per_rank((T // R, H)), per_rank((T // R, H))
        self.dWd, self.dWo = per_rank((H, F // R), f32), per_rank((H, H // R), f32)   # [out x in]
        self.dWug, self.dWqkv = per_rank((H, 2 * F // R), f32), per_rank((H, 3 * H // R), f32)

        P = {}
        # forward
        P["qkv"] = B.fo_plan("ag_gemm", R, T, 3 * H, H)
        P["o"] = B.fo_plan("gemm_rs", R, T, H, H, out_dtype="bf16")
        P["ug"] = B.fo_plan("ag_gemm", R, T, 2 * F, H)
        P["down"] = B.fo_plan("gemm_rs", R, T, H, F, out_dtype="bf16")
        # backward: data gradients
        P["down_dx"] = B.fo_plan("ag_gemm", R, T, F, H, w_layout="nk")
        P["ug_dx"] = B.fo_plan("gemm_rs", R, T, H, 2 * F, w_layout="nk", out_dtype="bf16")
        P["o_dx"] = B.fo_plan("ag_gemm", R, T, H, H, w_layout="nk")
        P["qkv_dx"] = B.fo_plan("gemm_rs", R, T, H, 3 * H, w_layout="nk", out_dtype="bf16")
        # backward: weight gradients (per-rank GEMMs, no collective)
        P["down_dw"] = B.fo_plan("dp_grad_rs", R, H, F // R, T)
        P["ug_dw"] = B.fo_plan("dp_grad_rs", R, H, 2 * F // R, T)
        P["o_dw"] = B.fo_plan("dp_grad_rs", R, H, H // R, T)
        P["qkv_dw"] = B.fo_plan("dp_grad_rs", R, H, 3 * H // R, T)
        self.plans = P
        self.ws = {}
        for k, p in P.items():
            self.ws[k] = torch.empty(B.fo_workspace_size(p), dtype=torch.uint8, device=dev)
            B.fo_workspace_init(p, self.ws[k])
        self.launches = 0

    def forward(self, stream=None):
        P, ws = self.plans, self.ws
        B.fo_ag_gemm(P["qkv"], self.x, self.Wqkv, self.y_qkv, self.Gx, ws["qkv"], stream)
        B.fo_gemm_rs(P["o"], self.attn, self.Wo, self.h, ws["o"], stream)
        B.fo_ag_gemm(P["ug"], self.h, self.Wug, self.y_ug, self.Gh, ws["ug"], stream)
        B.fo_gemm_rs(P["down"], self.act, self.Wd, self.y, ws["down"], stream)
        self.launches += 4

    def _weight_grad(self, key, G, shards, dY, dW, stream):
        """dW_r = AllGather(shards)^T . dY_r for every rank: from the
        gathered copy G when it was kept, else from the shards in place."""
        if G is not None:
            B.fo_gemm_partials(self.plans[key], G, dY, dW, self.ws[key], stream)
        else:
            B.fo_gemm_partials_sharded(self.plans[key], shards, dY, dW, self.ws[key], stream)

    def backward(self, stream=None):
        P, ws = self.plans, self.ws
        # down (row-parallel): dAct = AG(dy) . Wd^T, dWd^T = AG(dy)^T . act
        B.fo_ag_gemm(P["down_dx"], self.dy, self.Wd, self.d_act, self.G_dy, ws["down_dx"], stream)
        self._weight_grad("down_dw", self.G_dy, self.dy, self.act, self.dWd, stream)
        # up|gate (column-parallel): dh = RS(dug . Wug^T), dWug = AG(h)^T . dug
        B.fo_gemm_rs(P["ug_dx"], self.dug, self.Wug, self.d_h_from_ug, ws["ug_dx"], stream)
        self._weight_grad("ug_dw", self.Gh, self.h, self.dug, self.dWug, stream)
        # o (row-parallel): dAttn = AG(dh) . Wo^T, dWo^T = AG(dh)^T . attn
        B.fo_ag_gemm(P["o_dx"], self.dh, self.Wo, self.d_attn, self.G_dh, ws["o_dx"], stream)
        self._weight_grad("o_dw", self.G_dh, self.dh, self.attn, self.dWo, stream)
        # QKV (column-parallel): dx = RS(dqkv . Wqkv^T), dWqkv = AG(x)^T . dqkv
        B.fo_gemm_rs(P["qkv_dx"], self.dqkv, self.Wqkv, self.d_x, ws["qkv_dx"], stream)
        self._weight_grad("qkv_dw", self.Gx, self.x, self.dqkv, self.dWqkv, stream)
        self.launches += 8

    def status(self) -> List[int]:
        return [B.fo_status_query(p, self.ws[k])[0] for k, p in self.plans.items()]


def _on(stream):
    """torch's own work on a call's stream: None (the current one), a torch stream or a raw handle."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):   # (torch takes an external handle 0 for none)
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class Fp8AttentionBlock:
    """The attention half of a TP-SP layer with its projection in 8 bits, from the residual stream to the attention's
    output, and the way of the gradients back through what precedes the attention:

    forward
        norm      s = x + residual, n = rmsnorm(s); n in 8 bits with a scale for 128 columns   fo_rmsnorm
        QKV       Y_r = n . Wqkv_r^T, block-scaled 8-bit product, every rank in one launch    fo_gemm_fp8
        rotary    Y_r's Q and K turned by their positions, Q, K, V parted                     fo_rope
        attention + o projection + reduce-scatter                                             fo_attn_rs
    backward (dQ, dK, dV from the attention's own backward pass, which this framework does not have)
        rotary^-1 back into packed rows                                                       fo_rope
        QKV       dY_r in 8 bits, dn = sum_r dY_r . Wqkv_r (the weight's transposed copy)     fo_quant_fp8, fo_gemm_fp8,
                                                                                              fo_reduce_scatter_f32
                  (the products' partial sums by the unfused reduce kernel; the sum is rounded to bf16 by a torch copy)
        norm      dx (= d residual) with the residual path's gradient, dweight                fo_rmsnorm_bwd

    Q, K and V have the same heads, of 128 (fo_attn_rs has no others).
    The T tokens of the R ranks' shards lie back to back, so the norm is one call and its output is the all-gathered
    operand of every rank's product. The projections' weight gradients are not part of the block: they contract the
    tokens in bf16 (fo_gemm_partials_sharded), and the block keeps the norm's output in 8 bits alone. All of a call's
    work is on its stream, and what it returns are the block's own buffers, written again by the next call. Weights are
    given in bf16 ([3H/R x H] a rank, rows Q | K | V, the nn.Linear layout) and quantised by set_weights, once for each
    version of them."""

    def __init__(self, shape: LayerShape = LayerShape(), *, causal=True, eps=1e-6, rope_base=10000.0, device="cuda",
                 **rope):
        self.s = s = shape
        R, T, H = s.R, s.T, s.H
        if T % R or H % (R * 128):
            raise ValueError("T must be divisible by R, and H by R heads of 128")
        self.heads, self.causal = H // R // 128, causal
        width = H // R
        dev = torch.device(device)
        bf, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

        def new(*shp, dtype=bf):
            return torch.empty(shp, dtype=dtype, device=dev)

        def each(*shp, dtype=bf):
            return [new(*shp, dtype=dtype) for _ in range(R)]

        kb, nb = -(-H // 128), -(-3 * width // 128)
        self.norm = B.fo_norm_desc(H, eps=eps)
        self.qkv = B.fo_gemm_fp8_desc(3 * width, H, R=R)
        self.qkv_dx = B.fo_gemm_fp8_desc(H, 3 * width, R=R, out_dtype="f32")
        self.rope = B.fo_rope_desc(128, self.heads, self.heads, self.heads, R=R, base=rope_base, **rope)
        self.plan = B.fo_plan("gemm_rs", R, T, H, H, out_dtype="bf16")
        self.sum_plan = B.fo_plan("gemm_rs", R, T, H, H)          # its rows: the partial gradients' reduce-scatter
        # weights in 8 bits, as they are and transposed
        self.Wq, self.Wq_scale = each(3 * width, H, dtype=e4m3), each(nb, kb, dtype=f32)
        self.Wt, self.Wt_scale = each(H, 3 * width, dtype=e4m3), each(kb, nb, dtype=f32)
        # forward
        self.h, self.n8, self.n_scale, self.rstd = new(T, H), new(T, H, dtype=e4m3), new(T, kb, dtype=f32), new(T, dtype=f32)
        self.y_qkv = each(T, 3 * width)
        self.Q, self.K, self.V, self.O = (each(T, width) for _ in range(4))
        self.y = each(T // R, H)
        # backward
        self.d_qkv, self.d8, self.d_scale = each(T, 3 * width), each(T, 3 * width, dtype=e4m3), each(T, nb, dtype=f32)
        self.dn_part, self.dn_whole = each(T, H, dtype=f32), new(T, H, dtype=f32)
        self.dn = list(self.dn_whole.split(T // R))
        self.dn_rounded = new(T, H)
        self.dx, self.dweight = new(T, H), new(H, dtype=f32)
        self.ws_attn = new(B.fo_workspace_size(self.plan), dtype=torch.uint8)
        B.fo_workspace_init(self.plan, self.ws_attn)
        size = max(B.fo_gemm_fp8_workspace(self.qkv, T), B.fo_gemm_fp8_workspace(self.qkv_dx, T))
        self.ws = new(size, dtype=torch.uint8)
        B.fo_ops_workspace_init(self.ws)
        self.ws_norm = new(B.fo_rmsnorm_bwd_workspace(self.norm, T), dtype=torch.uint8)
        torch.cuda.current_stream(dev).synchronize()   # the workspaces are zeroed before a call on any other stream

    def set_weights(self, weight, Wqkv, Wo, stream=None):
        """The norm's weight [H], each rank's Wqkv [3H/R x H] and Wo [H/R x H], bf16."""
        width = self.s.H // self.s.R
        self.weight, self.Wo = weight, Wo
        B.fo_quant_fp8(3 * width, self.s.H, Wqkv, self.Wq, self.Wq_scale, self.Wt, self.Wt_scale, block_rows=128,
                       stream=stream)

    def _parts(self, packed):
        width = self.s.H // self.s.R
        return [[p[:, j * width:(j + 1) * width] for p in packed] for j in range(3)]

    def forward(self, x, residual=None, positions=None, stream=None):
        """x, residual [T x H] bf16 (the R token shards back to back), positions [T]; returns the R output shards.
        Five launches. h (the new residual) and rstd are kept for the backward pass."""
        T, R = self.s.T, self.s.R
        B.fo_rmsnorm(self.norm, T, [x], None if residual is None else [residual], self.weight, [self.h], None,
                     [self.n8], [self.n_scale], [self.rstd], stream)
        B.fo_gemm_fp8(self.qkv, T, [self.n8] * R, [self.n_scale] * R, self.Wq, self.Wq_scale, self.y_qkv, self.ws, stream)
        B.fo_rope(self.rope, T, positions, *self._parts(self.y_qkv), self.Q, self.K, self.V, stream=stream)
        B.fo_attn_rs(self.plan, self.Q, self.K, self.V, self.Wo, self.O, self.y, self.heads, self.causal, self.ws_attn,
                     stream)
        return self.y

    def backward(self, dQ, dK, dV, dh=None, positions=None, stream=None):
        """dQ, dK, dV [T x H/R] a rank, dh [T x H] the gradient that reaches the new residual by its own path; returns
        (dx, dweight), dx being the gradient of x and of the residual alike."""
        T, R, width = self.s.T, self.s.R, self.s.H // self.s.R
        B.fo_rope(self.rope, T, positions, dQ, dK, dV, *self._parts(self.d_qkv), inverse=True, stream=stream)
        B.fo_quant_fp8(T, 3 * width, self.d_qkv, self.d8, self.d_scale, stream=stream)
        B.fo_gemm_fp8(self.qkv_dx, T, self.d8, self.d_scale, self.Wt, self.Wt_scale, self.dn_part, self.ws, stream)
        B.fo_reduce_scatter_f32(self.sum_plan, self.dn_part, self.dn, stream)
        with _on(stream):
            self.dn_rounded.copy_(self.dn_whole)
        B.fo_rmsnorm_bwd(self.norm, T, [self.dn_rounded], None if dh is None else [dh], [self.h], self.weight, [self.rstd],
                         [self.dx], self.dweight, self.ws_norm, stream)
        return self.dx, self.dweight

    def status(self, stream=None) -> List[int]:
        """The status words once the stream's work so far is done (0: no device wait has run out)."""
        return [B.fo_status_query(self.plan, self.ws_attn, stream)[0], B.fo_ops_status_query(self.ws, stream)[0]]
