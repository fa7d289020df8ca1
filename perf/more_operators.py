"""The operators that serve a model from a paged cache of keys and values, as cases to be measured: appending to the cache with the
rotary positions on the way, and attention over the cache's pages, of one or a few new tokens a sequence and of whole prompts, with and
without a sliding window and first tokens that stay visible.

``own`` chooses what ``run`` calls: the plain forms below (elementary torch operations in 32 bits, angles in 64), or the library's calls.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TOP = 448.0                  # the largest e4m3 value
LEAST = 2.0 ** -126          # the smallest scale
BASE = 500000.0              # of the rotary frequencies


def listed():
    return [
        # A decode step's append: sixteen sequences' tokens with grouped-query heads. Latency.
        dict(name="append_decode", op="append", R=1, seqs=16, longest=8192, new=1, heads_q=32, heads_k=8, D=128, page=64, cache="bf16",
             rot=128, layout="half"),
        # A prompt of eight ranks, each with its own heads, from the projection's packed rows into the pages.
        dict(name="append_prompt", op="append", R=8, seqs=1, longest=8192, new=8192, heads_q=4, heads_k=4, D=128, page=64, cache="bf16",
             rot=128, layout="half"),
        # Ragged prompts into an 8-bit cache with small pages, half of each head rotated, in interleaved pairs.
        dict(name="append_8bit", op="append", R=1, seqs=7, longest=2500, new=1021, heads_q=32, heads_k=8, D=128, page=16, cache="e4m3",
             rot=64, layout="interleaved"),
        # A decode step of a few short conversations. Latency.
        dict(name="decode_short", op="attention", R=1, seqs=8, longest=512, new=1, heads_q=32, heads_k=8, D=128, page=64, cache="bf16",
             window=0, sinks=0, lse=False),
        # A decode step of a full batch of ragged contexts.
        dict(name="decode_batch", op="attention", R=1, seqs=64, longest=8192, new=1, heads_q=32, heads_k=8, D=128, page=64, cache="bf16",
             window=0, sinks=0, lse=False),
        # One conversation with a very long context: the cache's length is all the parallelism there is.
        dict(name="decode_long", op="attention", R=1, seqs=1, longest=131072, new=1, heads_q=32, heads_k=8, D=128, page=128, cache="bf16",
             window=0, sinks=0, lse=True),
        # The same kind of batch from an 8-bit cache.
        dict(name="decode_8bit", op="attention", R=1, seqs=32, longest=16384, new=1, heads_q=32, heads_k=8, D=128, page=32, cache="e4m3",
             window=0, sinks=0, lse=False),
        # Drafted tokens verified: up to five new ones a sequence, causal among themselves, two ranks, eight query heads a key head.
        dict(name="decode_drafted", op="attention", R=2, seqs=17, longest=4100, new=5, heads_q=16, heads_k=2, D=128, page=16, cache="bf16",
             window=0, sinks=0, lse=False),
        # A decode step far beyond the window, eight ranks; pages that the window has left are freed.
        dict(name="decode_window", op="attention", R=8, seqs=32, longest=32768, new=1, heads_q=4, heads_k=4, D=128, page=16, cache="bf16",
             window=1024, sinks=4, lse=False),
        # A whole prompt with a window and first tokens that stay visible.
        dict(name="prompt_window", op="attention", R=1, seqs=1, longest=8192, new=8192, heads_q=32, heads_k=8, D=128, page=64, cache="bf16",
             window=1024, sinks=4, lse=False),
        # A whole causal prompt of eight ranks, read back from the cache it has just been appended to.
        dict(name="prompt_causal", op="attention", R=8, seqs=1, longest=8192, new=8192, heads_q=4, heads_k=4, D=128, page=64, cache="bf16",
             window=0, sinks=0, lse=False),
        # Chunks of ragged prompts on cached prefixes, 8 bits, small heads and pages.
        dict(name="prompt_chunks_8bit", op="attention", R=1, seqs=5, longest=4111, new=1030, heads_q=16, heads_k=4, D=64, page=16,
             cache="e4m3", window=2000, sinks=64, lse=True),
    ]


def _spread(rng, lo, hi):
    """A whole number whose logarithm is spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    R = rng.choice((1, 1, 2, 4, 8))
    heads_k = rng.choice((1, 2, 4, 8))
    c = dict(R=R, heads_q=heads_k * rng.choice((1, 2, 3, 4, 7, 8, 16)), heads_k=heads_k, D=rng.choice((64, 128, 128)),
             page=rng.choice((16, 32, 64, 128)), cache=rng.choice(("bf16", "bf16", "e4m3")))
    kind = rng.choice(("append", "decode", "decode", "prompt"))
    if kind == "append":
        # At most the values of the largest listed append.
        most = 8192 * 8 * 12 * 128 // (R * (c["heads_q"] + 2 * heads_k) * c["D"])
        seqs = _spread(rng, 1, 256)
        new = _spread(rng, 1, max(1, min(8192, most // seqs)))
        return dict(c, op="append", seqs=seqs, new=new, longest=new + _spread(rng, 1, 2048), rot=rng.choice((c["D"], c["D"], c["D"] // 2)),
                    layout=rng.choice(("half", "interleaved")))
    windowed = rng.random() < 0.4
    c = dict(c, op="attention", window=_spread(rng, 16, 4096) if windowed else 0, sinks=rng.choice((0, 4, 64, 129)) if windowed else 0,
             lse=rng.random() < 0.3)
    if kind == "decode":
        # At most half of the cache that the largest listed batch reads.
        tokens = 64 * 8192 * 8 * 128 // (2 * R * heads_k * c["D"])
        longest = _spread(rng, 1, min(131072, tokens))
        seqs = _spread(rng, 1, max(1, min(256, tokens // longest)))
        return dict(c, seqs=seqs, longest=longest, new=min(longest, rng.choice((1, 1, 1, 2, 4, 7))))
    # At most a quarter of the (row, key) products of the largest listed prompt, counted without masks.
    pairs = 8 * 4 * 8192 * 8192 * 128 // (4 * R * c["heads_q"] * c["D"])
    seqs = _spread(rng, 1, 8)
    new = _spread(rng, 17, max(17, min(4096, int(math.sqrt(pairs / seqs)))))
    return dict(c, seqs=seqs, new=new, longest=new + rng.choice((0, _spread(rng, 1, max(1, min(8192, pairs // (seqs * new)))))))


def _lengths(case):
    """Tokens and new tokens of each sequence: the first has the most, the others are spread below it."""
    part = [i * 0.6180339887498949 % 1.0 for i in range(case["seqs"])]
    new = [max(1, int(case["new"] * (1 - 0.7 * p))) if 1 < case["new"] else 1 for p in part]
    return [max(n, int(case["longest"] * (1 - 0.75 * p))) for n, p in zip(new, part)], new


# ------------------------------------------------------------------ inputs

def _in_8_bits(x):
    """x [..., D] fp32 -> e4m3 values and one scale for each row of D."""
    scale = (x.abs().amax(dim=-1) / TOP).clamp(min=LEAST)
    return (x / scale[..., None]).to(E4M3), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    R, hq, hk, D, page, bf = c["R"], c["heads_q"], c["heads_k"], c["D"], c["page"], torch.bfloat16
    lengths, new = _lengths(case)
    c["rows"], c["max_new"], c["max_len"] = sum(new), max(new), max(lengths)
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    c["lengths"] = whole(lengths)
    # Without a list of first rows, every sequence has one new token.
    c["starts"] = whole([sum(new[:i]) for i in range(len(new) + 1)]) if c["max_new"] > 1 else None
    # Pages in no order, and the entries behind a sequence's end unused. Pages that lie wholly before the window of a sequence's first
    # new token and hold none of the tokens that stay visible are freed.
    cols = -(-c["max_len"] // page)
    c["pages"] = sum(-(-n // page) for n in lengths) + 3
    order, table, at = torch.randperm(c["pages"], generator=g, device="cuda").tolist(), [], 0
    for n, m in zip(lengths, new):
        held = -(-n // page)
        row = order[at:at + held] + [-1] * (cols - held)
        if c.get("window"):
            row = [-1 if (p + 1) * page <= n - m - c["window"] + 1 and p * page >= c["sinks"] else v for p, v in enumerate(row)]
        table.append(row)
        at += held
    c["table"] = whole(table)
    # Channels of different sizes, as keys have them.
    size = torch.exp(0.4 * torch.randn(D, generator=g, device="cuda"))
    shape = (c["pages"], hk, page, D)
    c["k_cache"] = [torch.randn(shape, generator=g, device="cuda", dtype=bf).mul_(size.to(bf)) for _ in range(R)]
    c["v_cache"] = [torch.randn(shape, generator=g, device="cuda", dtype=bf) for _ in range(R)]
    c["k_scale"] = c["v_scale"] = None
    if c["cache"] == "e4m3":
        c["k_cache"], c["k_scale"] = map(list, zip(*(_in_8_bits(x.float()) for x in c["k_cache"])))
        c["v_cache"], c["v_scale"] = map(list, zip(*(_in_8_bits(x.float()) for x in c["v_cache"])))
    if c["op"] == "append":
        # The projection's packed rows Q | K | V, the parts of each rank.
        heads = (hq, hk, hk)
        packed = [torch.randn(c["rows"], sum(heads) * D, generator=g, device="cuda", dtype=bf) for _ in range(R)]
        parts = [p.split([n * D for n in heads], dim=1) for p in packed]
        c["q"], c["k"], c["v"] = ([p[j] for p in parts] for j in range(3))
        c["q_out"] = [torch.empty(c["rows"], hq * D, dtype=bf, device="cuda") for _ in range(R)]
        i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
        c["frequencies"] = torch.exp(-math.log(BASE) * 2.0 * i / c["rot"])
    else:
        c["q"] = [torch.randn(c["rows"], hq * D, generator=g, device="cuda", dtype=bf) for _ in range(R)]
        c["o"] = [torch.empty(c["rows"], hq * D, dtype=bf, device="cuda") for _ in range(R)]
        c["lse_out"] = [torch.empty(c["rows"], hq, device="cuda") for _ in range(R)] if c["lse"] else None
    if own:
        from ag_gemm_gb300 import binding as B
        c["desc"] = B.fo_paged_desc(hq, hk, head_dim=D, R=R, page=page, cache=c["cache"], window=c.get("window", 0), sinks=c.get("sinks", 0))
        c["batch"] = B.fo_paged_batch(c["lengths"], c["table"], c["pages"], starts=c["starts"], max_new=c["max_new"])
        if c["op"] == "append":
            c["rope"] = B.fo_rope_desc(D, hq, hk, hk, R=R, rot_dim=c["rot"], layout=c["layout"], base=BASE)
        else:
            c["ws"] = torch.empty(B.fo_paged_attention_workspace(c["desc"], c["seqs"], c["rows"], c["max_new"]), dtype=torch.uint8, device="cuda")
            B.fo_ops_workspace_init(c["ws"])
    return c


# ------------------------------------------------------------------ one pass

def run(state):
    return _append(state) if state["op"] == "append" else _attention(state)


def _some(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _places(c):
    """The sequence of each row, and its token's number among the new ones and in the sequence."""
    row = torch.arange(c["rows"], device="cuda")
    if c["starts"] is None:
        return row, torch.zeros_like(row), c["lengths"].long() - 1
    starts = c["starts"].long()
    b = torch.searchsorted(starts, row, right=True) - 1
    i = row - starts[b]
    return b, i, c["lengths"].long()[b] - (starts[b + 1] - starts[b]) + i


def _append(c):
    if own:
        from ag_gemm_gb300 import binding as B
        B.fo_kv_append(c["desc"], c["rope"], c["batch"], c["rows"], c["q"], c["k"], c["v"], c["q_out"], c["k_cache"], c["v_cache"],
                       c["k_scale"], c["v_scale"])
        return _some(q=c["q_out"], k=c["k_cache"], v=c["v_cache"], k_scale=c["k_scale"], v_scale=c["v_scale"])
    rows, D, rot, page = c["rows"], c["D"], c["rot"], c["page"]
    b, _, pos = _places(c)
    at = c["table"][b, pos // page].long(), pos % page
    angle = torch.remainder(pos.double()[:, None] * c["frequencies"], 2 * math.pi)
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turned(x):
        v = x.reshape(rows, -1, D).float()
        out = v.clone()
        if c["layout"] == "half":
            a, b = v[..., : rot // 2], v[..., rot // 2: rot]
            out[..., : rot // 2], out[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = v[..., 0:rot:2], v[..., 1:rot:2]
            out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        return out

    def put(x, cache, scale):
        if scale is None:
            cache[at[0], :, at[1]] = x.to(cache.dtype)
        else:
            q, s = _in_8_bits(x)
            cache.view(torch.uint8)[at[0], :, at[1]] = q.view(torch.uint8)
            scale[at[0], :, at[1]] = s

    scales = lambda s: [None] * c["R"] if s is None else s  # noqa: E731
    [put(turned(x), cache, s) for x, cache, s in zip(c["k"], c["k_cache"], scales(c["k_scale"]))]
    [put(x.reshape(rows, -1, D).float(), cache, s) for x, cache, s in zip(c["v"], c["v_cache"], scales(c["v_scale"]))]
    q = [turned(x).to(x.dtype).view(rows, -1) for x in c["q"]]
    return _some(q=q, k=c["k_cache"], v=c["v_cache"], k_scale=c["k_scale"], v_scale=c["v_scale"])


def _attention(c):
    if own:
        from ag_gemm_gb300 import binding as B
        B.fo_paged_attention(c["desc"], c["batch"], c["rows"], c["q"], c["k_cache"], c["v_cache"], c["o"], c["ws"], c["k_scale"], c["v_scale"],
                             c["lse_out"])
        return _some(o=c["o"], lse=c["lse_out"])
    seqs, n, hk, D, page, dev = c["seqs"], c["max_new"], c["heads_k"], c["D"], c["page"], "cuda"
    group = c["heads_q"] // hk
    b, i, pos = _places(c)
    # Each sequence's new tokens side by side, the shorter ones' last places filled with some row.
    first = torch.zeros(seqs, dtype=torch.long, device=dev) if c["starts"] is None else c["starts"].long()[:-1]
    count = torch.ones_like(first) if c["starts"] is None else c["starts"].long()[1:] - first
    step = torch.arange(n, device=dev)
    row = torch.arange(seqs, device=dev)[:, None] if c["starts"] is None else (first[:, None] + step).clamp(max=c["rows"] - 1)
    p = (c["lengths"].long() - count)[:, None] + step
    table, whole = c["table"].clamp(min=0).long(), c["table"].shape[1] * page
    key = torch.arange(whole, device=dev)[None]
    if not c["window"]:
        sees = key[:, None] <= p[:, :, None]
    else:
        # The first tokens and those from the first one in the window of a sequence's first new token on.
        lo = (p[:, :1] - c["window"] + 1).clamp(min=0)
        early, near = key[:, :c["sinks"]].expand(seqs, -1), lo + key[:, : c["window"] + n - 1]
        key = torch.cat((early, near), dim=1)
        sees = torch.cat((early < lo, near < whole), dim=1)[:, None]
        sees = sees & (key[:, None] <= p[:, :, None]) & ((key[:, None] > p[:, :, None] - c["window"]) | (key[:, None] < c["sinks"]))
        key.clamp_(max=whole - 1)
        table = table.gather(1, key // page)
    hidden = ~sees[:, None, None]

    def read(cache, scale):
        if c["window"]:
            x = cache[table, :, key % page].float()
            return (x if scale is None else x.mul_(scale[table, :, key % page][..., None])).transpose(1, 2)
        x = cache[table].float()
        return (x if scale is None else x.mul_(scale[table][..., None])).transpose(1, 2).reshape(seqs, hk, whole, D)

    def one(q, k_cache, v_cache, k_scale, v_scale):
        qs = (q.float() / math.sqrt(D)).view(-1, hk, group, D)[row].permute(0, 2, 3, 1, 4)     # sequence, key head, head of the group, token
        s = torch.matmul(qs.reshape(seqs, hk, group * n, D), read(k_cache, k_scale).transpose(2, 3)).view(seqs, hk, group, n, -1)
        s.masked_fill_(hidden, -math.inf)
        m = s.amax(dim=-1, keepdim=True)
        s = s.sub_(m).exp_()
        total = s.sum(dim=-1, keepdim=True)
        o = torch.matmul(s.view(seqs, hk, group * n, -1), read(v_cache, v_scale)).view(seqs, hk, group, n, D) / total
        lse = (m + total.log())[..., 0]
        return o[b, :, :, i].reshape(c["rows"], -1).to(q.dtype), lse[b, :, :, i].reshape(c["rows"], -1)

    no = [None] * c["R"]
    got = [one(*x) for x in zip(c["q"], c["k_cache"], c["v_cache"], c["k_scale"] or no, c["v_scale"] or no)]
    return _some(o=[o for o, _ in got], lse=[x for _, x in got] if c["lse"] else None)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    R, hq, hk, D = c["R"], c["heads_q"], c["heads_k"], c["D"]
    lengths, new = _lengths(c)
    rows, seqs = sum(new), c["seqs"]
    kept = 2 * D * 2 if c["cache"] == "bf16" else 2 * (D + 4)      # a token's key and value of one head, in the cache
    lists = 4 * (2 * seqs + 1)
    if c["op"] == "append":
        return {"bytes": R * rows * ((2 * hq + 2 * hk) * D * 2 + hk * kept) + lists + 4 * rows, "flops": 3 * R * rows * (hq + hk) * c["rot"]}
    read, pairs = 0, 0
    for n, m in zip(lengths, new):
        w, s = c["window"] or n, c["sinks"]
        first = max(0, n - m - w + 1)                              # the first key in the window of the first new token
        read += n - first + min(s, first)
        for p in range(n - m, n):
            lo = max(0, p - w + 1)
            pairs += p + 1 - lo + min(s, lo)
    return {"bytes": R * (rows * hq * (2 * D * 2 + (4 if c["lse"] else 0)) + read * hk * kept) + lists + 4 * sum(-(-n // c["page"]) for n in lengths),
            "flops": 4 * D * R * hq * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits (numbers as they are before they are stored in their type)

def exact(case, seed):
    c = prepare(case, seed)
    lengths, new = _lengths(case)
    hq, hk, D, page, table = c["heads_q"], c["heads_k"], c["D"], c["page"], c["table"].tolist()
    where = [(b, n - m + i) for b, (n, m) in enumerate(zip(lengths, new)) for i in range(m)]
    if c["op"] == "append":
        pos = torch.tensor([p for _, p in where], dtype=torch.float64, device="cuda")
        # Pairs as complex numbers, turned by exp(i angle).
        angle = torch.outer(pos, c["frequencies"])
        turn, rot = torch.polar(torch.ones_like(angle), angle)[:, None, :], c["rot"]
        pages = torch.tensor([table[b][p // page] for b, p in where], device="cuda")
        slots = torch.tensor([p % page for _, p in where], device="cuda")

        def turned(x):
            v = x.double().reshape(c["rows"], -1, D)
            head = v[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["layout"] == "half" else v[..., :rot].unflatten(-1, (rot // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
            z = (z.transpose(-1, -2) if c["layout"] == "half" else z).reshape(c["rows"], -1, rot)
            return torch.cat((z, v[..., rot:]), dim=-1)

        def kept(x, cache, scale):
            out = cache.double()
            if scale is None:
                out[pages, :, slots] = x
                return out, None
            s = torch.maximum(x.abs().max(dim=-1).values / TOP, torch.tensor(LEAST, dtype=torch.float64, device="cuda"))
            scales = scale.double()
            out[pages, :, slots], scales[pages, :, slots] = x / s[..., None], s
            return out, scales

        no = [None] * c["R"]
        k = [kept(turned(x), cache, s) for x, cache, s in zip(c["k"], c["k_cache"], c["k_scale"] or no)]
        v = [kept(x.double().reshape(c["rows"], -1, D), cache, s) for x, cache, s in zip(c["v"], c["v_cache"], c["v_scale"] or no)]
        scaled = c["cache"] == "e4m3"
        return _some(q=[turned(x).reshape(c["rows"], -1) for x in c["q"]], k=[x for x, _ in k], v=[x for x, _ in v],
                     k_scale=[s for _, s in k] if scaled else None, v_scale=[s for _, s in v] if scaled else None)
    # Head by head of each sequence, over the keys that one of its new tokens sees.
    outs, sums = [], []
    for r in range(c["R"]):
        o = torch.empty(c["rows"], hq, D, dtype=torch.float64, device="cuda")
        lse = torch.empty(c["rows"], hq, dtype=torch.float64, device="cuda")
        at = 0
        for b, (n, m) in enumerate(zip(lengths, new)):
            key = torch.arange(n, device="cuda")
            if c["window"]:
                key = key[(key > n - m - c["window"]) | (key < c["sinks"])]
            page_of, slot = c["table"][b].long()[key // page], key % page
            kv = []
            for cache, scale in ((c["k_cache"], c["k_scale"]), (c["v_cache"], c["v_scale"])):
                x = cache[r][page_of, :, slot].double()
                kv.append(x if scale is None else x * scale[r][page_of, :, slot, None].double())
            for lo in range(0, m, 2048):
                rows = slice(at + lo, at + min(m, lo + 2048))
                pos = torch.arange(n - m + lo, n - m + min(m, lo + 2048), device="cuda")[:, None]
                hidden = key > pos
                if c["window"]:
                    hidden |= (key <= pos - c["window"]) & (key >= c["sinks"])
                for h in range(hq):
                    j = h // (hq // hk)
                    s = (c["q"][r][rows, h * D:(h + 1) * D].double() @ kv[0][:, j].t()) * D ** -0.5
                    s = s.masked_fill(hidden, -math.inf)
                    lse[rows, h] = torch.logsumexp(s, dim=1)
                    o[rows, h] = torch.exp(s - lse[rows, h, None]) @ kv[1][:, j]
            at += m
        outs.append(o.reshape(c["rows"], -1))
        sums.append(lse)
    return _some(o=outs, lse=sums if c["lse"] else None)
