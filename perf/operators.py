"""The operators between a layer's residual stream and its attention, as cases to be measured: RMSNorm with the residual's addition,
quantisation to 8 bits, the product of 8-bit matrices with a scale for each block of 128, and rotary positions.

``own`` chooses what ``run`` calls: the plain forms below (elementary torch operations in 32 bits, angles in 64), or the library's calls.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TOP = 448.0                  # the largest e4m3 value
LEAST = 2.0 ** -126          # the smallest scale
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # A decode step's norm: a few sequences' tokens, the residual added, 8 bits for the projection that follows. Latency.
        dict(name="norm_decode", op="norm", rows=8, H=4096, dtype="bf16", residual=True, out="q"),
        # The norm before the QKV projection of a whole prompt.
        dict(name="norm_prefill", op="norm", rows=8192, H=4096, dtype="bf16", residual=True, out="q"),
        # An fp32 model of an odd width: rows without 16-byte alignment.
        dict(name="norm_odd_f32", op="norm", rows=1021, H=1357, dtype="f32", residual=False, out="y"),
        # The training step's backward pass of the norm: dx with the residual's own gradient added, and the weight's gradient.
        dict(name="norm_backward", op="norm_bwd", rows=8192, H=4096, dtype="bf16", residual=True),
        # Activations and upstream gradients into 8 bits, one scale for 128 values of a row.
        dict(name="quant_rows", op="quant", rows=8192, cols=4096, dtype="bf16", block_rows=1),
        # A weight after the optimiser's step: one scale for each 128 x 128 block, and the transposed copy for the input gradient.
        dict(name="quant_weight", op="quant", rows=12288, cols=4096, dtype="bf16", block_rows=128),
        # The QKV projection of one decode step: the weight is streamed for four tokens.
        dict(name="gemm_decode", op="gemm", R=1, M=4, N=12288, K=4096, out="bf16"),
        # A short prompt on a narrow layer: ragged rows and columns, a last block of the reduction that is not full.
        dict(name="gemm_ragged", op="gemm", R=1, M=333, N=1000, K=1744, out="f32"),
        # The QKV projection of a whole prompt, eight ranks' column slices in one call.
        dict(name="gemm_prefill", op="gemm", R=8, M=8192, N=1536, K=4096, out="bf16"),
        # A decode step of grouped-query attention: 32 query heads, 8 key heads, far positions.
        dict(name="rope_decode", op="rope", R=1, rows=16, heads_q=32, heads_k=8, heads_v=8, D=128, rot=128, layout="half", dtype="bf16",
             inverse=False, scaling="wavelength", far=131072),
        # A prompt's packed QKV rows of eight ranks into the attention's Q, K and V.
        dict(name="rope_prefill", op="rope", R=8, rows=8192, heads_q=4, heads_k=4, heads_v=4, D=128, rot=128, layout="half", dtype="bf16",
             inverse=False, scaling="none", far=8192),
        # The gradient's way back through interleaved pairs on half of the head, positions scaled for a long context, fp32.
        dict(name="rope_backward", op="rope", R=1, rows=4095, heads_q=16, heads_k=4, heads_v=4, D=128, rot=64, layout="interleaved",
             dtype="f32", inverse=True, scaling="parts", far=1000000),
    ]


def _spread(rng, lo, hi):
    """A whole number whose logarithm is spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "quant", "gemm", "gemm", "rope"))
    if op in ("norm", "norm_bwd"):
        H = _spread(rng, 64, 16384)
        if rng.random() < 0.6:
            H = max(64, H // 128 * 128)
        rows = _spread(rng, 1, max(1, min(16384, 8192 * 4096 // H)))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        rows = rows if dtype == "bf16" else max(1, rows // 2)
        c = dict(op=op, rows=rows, H=H, dtype=dtype, residual=rng.random() < 0.6)
        return dict(c, out=rng.choice(("y", "q", "both"))) if op == "norm" else c
    if op == "quant":
        cols = _spread(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = max(64, cols // 128 * 128)
        rows = _spread(rng, 1, max(1, min(28672, 12288 * 4096 // cols)))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        return dict(op=op, rows=rows if dtype == "bf16" else max(1, rows // 2), cols=cols, dtype=dtype, block_rows=rng.choice((1, 128)))
    if op == "gemm":
        R = rng.choice((1, 1, 2, 4, 8))
        K = max(16, _spread(rng, 128, 14336) // 16 * 16)
        N = _spread(rng, 64, 28672 // R)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        M = _spread(rng, 1, max(1, min(8192, 8192 * 12288 * 4096 // (R * N * K))))
        return dict(op=op, R=R, M=M, N=N, K=K, out=rng.choice(("bf16", "bf16", "f32")))
    R = rng.choice((1, 1, 2, 4, 8))
    D = rng.choice((64, 80, 96, 128, 128, 192, 256))
    rot = rng.choice((D, D, D // 2, D // 4))
    heads_k = rng.choice((1, 2, 4, 8))
    heads_q = heads_k * rng.choice((1, 2, 4, 8))
    heads_v = rng.choice((0, heads_k))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    most = 8192 * 8 * 12 * 128 // (R * (heads_q + heads_k + heads_v) * D)
    rows = _spread(rng, 1, max(1, min(16384, most if dtype == "bf16" else most // 2)))
    return dict(op=op, R=R, rows=rows, heads_q=heads_q, heads_k=heads_k, heads_v=heads_v, D=D, rot=rot, layout=rng.choice(("half", "interleaved")),
                dtype=dtype, inverse=rng.random() < 0.4, scaling=rng.choice(("none", "linear", "wavelength", "parts")),
                far=rng.choice((4096, 131072, 1000000)))


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows_in_8_bits(x):
    """x [rows, cols] fp32 -> e4m3 values and one scale for 128 columns of a row."""
    rows, cols = x.shape
    groups = -(-cols // 128)
    padded = torch.zeros(rows, groups * 128, device=x.device)
    padded[:, :cols] = x
    padded = padded.view(rows, groups, 128)
    scale = (padded.abs().amax(dim=2) / TOP).clamp(min=LEAST)
    return (padded / scale[:, :, None]).to(E4M3).view(rows, groups * 128)[:, :cols].contiguous(), scale


def _blocks_in_8_bits(x):
    """x [rows, cols] fp32 -> e4m3 values and one scale for each 128 x 128 block."""
    rows, cols = x.shape
    up, across = -(-rows // 128), -(-cols // 128)
    padded = torch.zeros(up * 128, across * 128, device=x.device)
    padded[:rows, :cols] = x
    padded = padded.view(up, 128, across, 128)
    scale = (padded.abs().amax(dim=(1, 3)) / TOP).clamp(min=LEAST)
    return (padded / scale[:, None, :, None]).to(E4M3).view(up * 128, across * 128)[:rows, :cols].contiguous(), scale


#: The scalings of the rotary frequencies: f is the unscaled one in radians, the arguments what a model's configuration gives.
ROPE_BASE = 500000.0
STRETCH = 8.0                       # how much longer the context is than the one trained on
TRAINED = 8192                      # the context trained on
SLOW, FAST = 1.0, 4.0               # "wavelength": turns in the trained context below which f is divided, above which it stays
FEW, MANY = 1.0, 32.0               # "parts": the same borders, the mix linear in the pair's index


def _frequencies(rot, scaling):
    """Radians a position for each pair, in 64 bits, and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = torch.exp(-math.log(ROPE_BASE) * 2.0 * i / rot)
    if scaling == "linear":
        return f / STRETCH, 1.0
    if scaling == "wavelength":
        keep = ((TRAINED * f / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
        return keep * f + (1 - keep) * f / STRETCH, 1.0
    if scaling == "parts":
        at = [rot * math.log(TRAINED / (2 * math.pi * n)) / (2 * math.log(ROPE_BASE)) for n in (MANY, FEW)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return keep * f + (1 - keep) * f / STRETCH, 0.1 * math.log(STRETCH) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] in ("norm", "norm_bwd"):
        t, rows, H = TYPES[c["dtype"]], c["rows"], c["H"]
        # A residual stream: channels of different sizes, some rows far larger than others.
        size = torch.exp(0.5 * _randn(g, H))[None, :] * torch.exp(0.7 * _randn(g, rows))[:, None]
        c["weight"] = (1 + 0.2 * _randn(g, H)).to(t)
        f32 = dict(dtype=torch.float32, device="cuda")
        if c["op"] == "norm":
            c["x"] = (_randn(g, rows, H) * size).to(t)
            c["res"] = (_randn(g, rows, H) * size).to(t) if c["residual"] else None
            c["h_out"] = torch.empty_like(c["x"]) if c["residual"] else None
            c["y_out"] = torch.empty_like(c["x"]) if c["out"] != "q" else None
            c["q_out"] = torch.empty(rows, H, dtype=E4M3, device="cuda") if c["out"] != "y" else None
            c["scale_out"] = torch.empty(rows, -(-H // 128), **f32) if c["out"] != "y" else None
            c["rstd_out"] = torch.empty(rows, **f32)
        else:
            c["h"] = (_randn(g, rows, H) * size).to(t)
            c["rstd"] = torch.rsqrt(c["h"].float().square().mean(dim=1) + EPS)
            c["dy"] = (1e-2 * _randn(g, rows, H)).to(t)
            c["dh"] = (1e-2 * _randn(g, rows, H)).to(t) if c["residual"] else None
            c["dx_out"], c["dw_out"] = torch.empty_like(c["h"]), torch.empty(H, **f32)
        if own:
            from ag_gemm_gb300 import binding as B
            c["desc"] = B.fo_norm_desc(H, dtype=c["dtype"], eps=EPS)
            if c["op"] == "norm_bwd":
                c["ws"] = torch.empty(B.fo_rmsnorm_bwd_workspace(c["desc"], rows), dtype=torch.uint8, device="cuda")
    elif c["op"] == "quant":
        rows, cols = c["rows"], c["cols"]
        spread = 0.5 if c["block_rows"] == 128 else 1.0
        c["x"] = (_randn(g, rows, cols) * torch.exp(spread * _randn(g, rows))[:, None]).to(TYPES[c["dtype"]])
        up, across = -(-rows // c["block_rows"]), -(-cols // 128)
        c["q_out"] = torch.empty(rows, cols, dtype=E4M3, device="cuda")
        c["scale_out"] = torch.empty(up, across, device="cuda")
        c["qt_out"] = torch.empty(cols, rows, dtype=E4M3, device="cuda") if c["block_rows"] == 128 else None
        c["scale_t_out"] = torch.empty(across, up, device="cuda") if c["block_rows"] == 128 else None
    elif c["op"] == "gemm":
        R, M, N, K = c["R"], c["M"], c["N"], c["K"]
        # One matrix of tokens that every rank reads, each rank's slice of the weight.
        c["A"], c["sA"] = _rows_in_8_bits(_randn(g, M, K) * torch.exp(0.5 * _randn(g, M))[:, None])
        c["W"], c["sW"] = map(list, zip(*(_blocks_in_8_bits(0.02 * _randn(g, N, K)) for _ in range(R))))
        c["Y"] = [torch.empty(M, N, dtype=TYPES[c["out"]], device="cuda") for _ in range(R)]
        if own:
            from ag_gemm_gb300 import binding as B
            c["desc"] = B.fo_gemm_fp8_desc(N, K, R=R, out_dtype=c["out"])
            c["ws"] = torch.empty(B.fo_gemm_fp8_workspace(c["desc"], M), dtype=torch.uint8, device="cuda")
            B.fo_ops_workspace_init(c["ws"])
    else:
        R, rows, D, t = c["R"], c["rows"], c["D"], TYPES[c["dtype"]]
        heads = (c["heads_q"], c["heads_k"], c["heads_v"])
        packed = lambda: torch.empty(rows, sum(heads) * D, dtype=t, device="cuda")  # noqa: E731
        parted = lambda: [torch.empty(rows, n * D, dtype=t, device="cuda") if n else None for n in heads]  # noqa: E731
        # Forward: packed rows in, Q, K and V out. The gradient goes the other way.
        ins = [parted() if c["inverse"] else packed().split([n * D for n in heads], dim=1) for _ in range(R)]
        outs = [packed().split([n * D for n in heads], dim=1) if c["inverse"] else parted() for _ in range(R)]
        c["ins"], c["outs"] = [[[p[j] for p in side] for j in range(3)] for side in (ins, outs)]
        for x in (x for part in c["ins"] for x in part if x is not None):
            x.copy_(_randn(g, *x.shape))
        c["positions"] = torch.randint(0, c["far"], (rows,), generator=g, device="cuda")
        f, c["factor"] = _frequencies(c["rot"], c["scaling"])
        c["frequencies"] = f.cuda()
        if own:
            from ag_gemm_gb300 import binding as B
            extra = {"none": {}, "linear": dict(stretch=STRETCH), "wavelength": dict(stretch=STRETCH, trained=TRAINED, slow=SLOW, fast=FAST),
                     "parts": dict(stretch=STRETCH, trained=TRAINED, slow=FEW, fast=MANY)}[c["scaling"]]
            c["desc"] = B.fo_rope_desc(D, *heads, R=R, rot_dim=c["rot"], layout=c["layout"], dtype=c["dtype"], base=ROPE_BASE,
                                       scaling=c["scaling"], **extra)
    return c


# ------------------------------------------------------------------ one pass

def run(state):
    return {"norm": _norm, "norm_bwd": _norm_bwd, "quant": _quant, "gemm": _gemm, "rope": _rope}[state["op"]](state)


def _some(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _norm(c):
    if own:
        from ag_gemm_gb300 import binding as B
        one = lambda v: None if v is None else [v]  # noqa: E731
        B.fo_rmsnorm(c["desc"], c["rows"], [c["x"]], one(c["res"]), c["weight"], one(c["h_out"]), one(c["y_out"]), one(c["q_out"]),
                     one(c["scale_out"]), [c["rstd_out"]])
        return _some(h=c["h_out"], y=c["y_out"], q=c["q_out"], scale=c["scale_out"], rstd=c["rstd_out"])
    s = c["x"].float()
    if c["res"] is not None:
        s = s + c["res"].float()
    rstd = torch.rsqrt(s.square().mean(dim=1) + EPS)
    n = s * rstd[:, None] * c["weight"].float()
    q, scale = _rows_in_8_bits(n) if c["out"] != "y" else (None, None)
    return _some(h=s.to(c["x"].dtype) if c["residual"] else None, y=n.to(c["x"].dtype) if c["out"] != "q" else None, q=q, scale=scale, rstd=rstd)


def _norm_bwd(c):
    if own:
        from ag_gemm_gb300 import binding as B
        B.fo_rmsnorm_bwd(c["desc"], c["rows"], [c["dy"]], None if c["dh"] is None else [c["dh"]], [c["h"]], c["weight"], [c["rstd"]],
                         [c["dx_out"]], c["dw_out"], c["ws"])
        return {"dx": c["dx_out"], "dw": c["dw_out"]}
    dy, h, rstd = c["dy"].float(), c["h"].float(), c["rstd"][:, None]
    u = dy * c["weight"].float()
    dx = rstd * u - h * (rstd ** 3 * (u * h).mean(dim=1, keepdim=True))
    if c["dh"] is not None:
        dx = dx + c["dh"].float()
    return {"dx": dx.to(c["h"].dtype), "dw": (dy * h * rstd).sum(dim=0)}


def _quant(c):
    if own:
        from ag_gemm_gb300 import binding as B
        one = lambda v: None if v is None else [v]  # noqa: E731
        B.fo_quant_fp8(c["rows"], c["cols"], [c["x"]], [c["q_out"]], [c["scale_out"]], one(c["qt_out"]), one(c["scale_t_out"]),
                       block_rows=c["block_rows"])
        return _some(q=c["q_out"], scale=c["scale_out"], qt=c["qt_out"], scale_t=c["scale_t_out"])
    if c["block_rows"] == 1:
        q, scale = _rows_in_8_bits(c["x"].float())
        return {"q": q, "scale": scale}
    q, scale = _blocks_in_8_bits(c["x"].float())
    return {"q": q, "scale": scale, "qt": q.t().contiguous(), "scale_t": scale.t().contiguous()}


def _gemm(c):
    R = c["R"]
    if own:
        from ag_gemm_gb300 import binding as B
        B.fo_gemm_fp8(c["desc"], c["M"], [c["A"]] * R, [c["sA"]] * R, c["W"], c["sW"], c["Y"], c["ws"])
        return c["Y"]
    K, N = c["K"], c["N"]
    a = c["A"].float() * c["sA"].repeat_interleave(128, dim=1)[:, :K]
    return [(a @ (w.float() * s.repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)[:, :K]).t()).to(TYPES[c["out"]])
            for w, s in zip(c["W"], c["sW"])]


def _rope(c):
    if own:
        from ag_gemm_gb300 import binding as B
        B.fo_rope(c["desc"], c["rows"], c["positions"], *c["ins"], *c["outs"], inverse=c["inverse"])
        return [[x for x in part if x is not None and x.numel()] for part in c["outs"]]
    rows, D, rot = c["rows"], c["D"], c["rot"]
    angle = torch.remainder(c["positions"].double()[:, None] * c["frequencies"], 2 * math.pi)
    cos, sin = (angle.cos() * c["factor"]).float()[:, None, :], (angle.sin() * c["factor"]).float()[:, None, :]
    if c["inverse"]:
        sin = -sin

    def turned(x):
        v = x.reshape(rows, -1, D).float()
        out = v.clone()
        if c["layout"] == "half":
            a, b = v[..., : rot // 2], v[..., rot // 2: rot]
            out[..., : rot // 2], out[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = v[..., 0:rot:2], v[..., 1:rot:2]
            out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        return out.to(x.dtype).view(rows, -1)

    q, k, v = c["ins"]
    return [[turned(x) for x in q], [turned(x) for x in k], [x.clone() for x in v if x is not None and x.numel()]]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        e = 2 if c["dtype"] == "bf16" else 4
        n, groups = c["rows"] * c["H"], c["rows"] * -(-c["H"] // 128)
        if c["op"] == "norm_bwd":
            return {"bytes": n * e * (4 if c["residual"] else 3) + 4 * c["rows"] + (e + 4) * c["H"], "flops": 10 * n}
        b = n * e * (3 if c["residual"] else 1) + (n * e if c["out"] != "q" else 0) + (n + 4 * groups if c["out"] != "y" else 0)
        return {"bytes": b + e * c["H"] + 4 * c["rows"], "flops": 6 * n}
    if c["op"] == "quant":
        n, e = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        scales = 4 * -(-c["rows"] // c["block_rows"]) * -(-c["cols"] // 128)
        return {"bytes": n * e + (n + scales) * (2 if c["block_rows"] == 128 else 1), "flops": 3 * n}
    if c["op"] == "gemm":
        R, M, N, K = c["R"], c["M"], c["N"], c["K"]
        k = -(-K // 128)
        return {"bytes": M * (K + 4 * k) + R * (N * K + 4 * k * -(-N // 128) + M * N * (2 if c["out"] == "bf16" else 4)), "flops": 2 * R * M * N * K}
    n = c["R"] * c["rows"] * (c["heads_q"] + c["heads_k"] + c["heads_v"]) * c["D"]
    turned = c["R"] * c["rows"] * (c["heads_q"] + c["heads_k"]) * c["rot"]
    return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 8 * c["rows"], "flops": 3 * turned}


# ------------------------------------------------------------------ the definitions in 64 bits (numbers as they are before they are stored in their type)

def _exact_scales(n, up, across=128):
    """max(largest magnitude / 448, 2^-126) of each up x across block, and that number for each value."""
    rows, cols = n.shape
    blocks = torch.nn.functional.pad(n.abs(), (0, -cols % across, 0, -rows % up)).unfold(0, up, up).unfold(1, across, across)
    scale = torch.maximum(blocks.flatten(2).max(dim=2).values / TOP, torch.tensor(LEAST, dtype=torch.float64, device=n.device))
    r, k = torch.arange(rows, device=n.device) // up, torch.arange(cols, device=n.device) // across
    return scale, scale[r][:, k]


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "norm":
        s = c["x"].double()
        if c["residual"]:
            s += c["res"].double()
        rstd = 1 / torch.sqrt((s * s).sum(dim=1) / c["H"] + EPS)
        n = torch.einsum("rh,r,h->rh", s, rstd, c["weight"].double())
        out = dict(h=s if c["residual"] else None, y=n if c["out"] != "q" else None, rstd=rstd, q=None, scale=None)
        if c["out"] != "y":
            out["scale"], each = _exact_scales(n, 1)
            out["q"] = n / each
        return _some(**out)
    if c["op"] == "norm_bwd":
        h, dy, w, r = c["h"].double(), c["dy"].double(), c["weight"].double(), c["rstd"].double()
        along = torch.einsum("rh,rh,h->r", dy, h, w) / c["H"]
        dx = dy * w * r[:, None] - h * (along * r ** 3)[:, None]
        return {"dx": dx + c["dh"].double() if c["residual"] else dx, "dw": torch.einsum("rh,rh,r->h", dy, h, r)}
    if c["op"] == "quant":
        x = c["x"].double()
        scale, each = _exact_scales(x, c["block_rows"])
        q = x / each
        return {"q": q, "scale": scale} if c["block_rows"] == 1 else {"q": q, "scale": scale, "qt": q.t().contiguous(), "scale_t": scale.t().contiguous()}
    if c["op"] == "gemm":
        # Block by block of the reduction: each block's product has its own scales.
        got = []
        for w, s in zip(c["W"], c["sW"]):
            y = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
            for b in range(-(-c["K"] // 128)):
                k = slice(128 * b, 128 * b + 128)
                scaled = c["A"][:, k].double() * c["sA"][:, b, None].double()
                y.addmm_(scaled, (w[:, k].double() * s[torch.arange(c["N"], device="cuda") // 128, b, None].double()).t())
            got.append(y)
        return got
    # Pairs as complex numbers, turned by exp(i angle).
    rows, D, rot = c["rows"], c["D"], c["rot"]
    angle = torch.outer(c["positions"].double(), c["frequencies"]) * (-1 if c["inverse"] else 1)
    turn = torch.polar(torch.full_like(angle, c["factor"]), angle)[:, None, :]

    def turned(x):
        v = x.double().reshape(rows, -1, D)
        head = v[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["layout"] == "half" else v[..., :rot].unflatten(-1, (rot // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
        z = (z.transpose(-1, -2) if c["layout"] == "half" else z).reshape(rows, -1, rot)
        return torch.cat((z, v[..., rot:]), dim=-1).reshape(rows, -1)

    q, k, v = c["ins"]
    return [[turned(x) for x in q], [turned(x) for x in k], [x.double() for x in v if x is not None and x.numel()]]
