"""The decoder-layer operators around the weight stream, as measured cases.

Four operators: attention of new tokens over a paged key-value cache
(``attn``), rotary positions with the append to that cache (``append``), the
norms around a block with its gate and residual scale (``norm``), and a
mixture-of-experts layer for a few tokens (``moe``).  With ``own`` false,
``run`` computes them in plain 32-bit torch; with ``own`` true it calls the
library's entry points.  ``exact`` evaluates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one user's first tokens: one sequence, a short cache, the 4096-wide decoder's heads
        {"name": "attn one short f16", "op": "attn", "type": "f16", "batch": 1, "q_len": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "len_min": 100, "len_max": 100,
         "window": 0, "sinks": 0},
        # a serving batch of ragged lengths on the 1536-wide decoder's heads
        {"name": "attn ragged batch f16", "op": "attn", "type": "f16", "batch": 16, "q_len": 1,
         "heads": 12, "kv_heads": 2, "head_dim": 128, "page": 16, "len_min": 1, "len_max": 8191,
         "window": 0, "sinks": 0},
        # one long document: the cache is the whole cost
        {"name": "attn one long bf16", "op": "attn", "type": "bf16", "batch": 1, "q_len": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "len_min": 200001,
         "len_max": 200001, "window": 0, "sinks": 0},
        # draft tokens verified under a sliding window with sink tokens, small heads
        {"name": "attn verify window bf16", "op": "attn", "type": "bf16", "batch": 8, "q_len": 8,
         "heads": 32, "kv_heads": 8, "head_dim": 64, "page": 16, "len_min": 3000,
         "len_max": 40000, "window": 4096, "sinks": 4},
        # one new token of one sequence
        {"name": "append one f16", "op": "append", "type": "f16", "batch": 1, "q_len": 1,
         "heads": 12, "kv_heads": 2, "head_dim": 128, "rot": 128, "page": 16, "len_min": 1000,
         "len_max": 1000, "inter": 0},
        # draft tokens of a serving batch, rotary part of each head in interleaved pairs
        {"name": "append batch bf16", "op": "append", "type": "bf16", "batch": 256, "q_len": 8,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 64, "page": 16, "len_min": 17,
         "len_max": 700, "inter": 1},
        # one token's residual add and the next block's norm, 1536-wide decoder
        {"name": "norm one f16", "op": "norm", "type": "f16", "rows": 1, "width": 1536,
         "layer": 0, "post": 0, "gate": 0, "h32": 0},
        # many rows, norms on both sides of the block with a gate, wide residual in fp32
        {"name": "norm many bf16", "op": "norm", "type": "bf16", "rows": 4096, "width": 4096,
         "layer": 0, "post": 1, "gate": 1, "h32": 1},
        # one token through many small experts
        {"name": "moe one f16", "op": "moe", "type": "f16", "int4": 0, "tokens": 1,
         "hidden": 2048, "inter": 1024, "experts": 64, "top_k": 8},
        # a few draft tokens, int4 experts
        {"name": "moe few int4", "op": "moe", "type": "f16", "int4": 1, "tokens": 4,
         "hidden": 4096, "inter": 1536, "experts": 128, "top_k": 8},
        # one token, two of eight wide int4 experts (the 4096-wide decoder's matrices)
        {"name": "moe one wide int4", "op": "moe", "type": "f16", "int4": 1, "tokens": 1,
         "hidden": 4096, "inter": 14336, "experts": 8, "top_k": 2},
        # the most tokens, wide bf16 experts
        {"name": "moe sixteen wide bf16", "op": "moe", "type": "bf16", "int4": 0, "tokens": 16,
         "hidden": 4096, "inter": 14336, "experts": 8, "top_k": 2},
    ]


def _log(rng, lo, hi, unit=1):
    """A multiple of unit, spread over the logarithm of [lo, hi] units."""
    n = unit * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + unit if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "norm", "moe", "moe"])
    kind = rng.choice(["f16", "bf16"])
    heads, kv_heads = rng.choice([(12, 2), (32, 8), (16, 16), (28, 4), (24, 1), (40, 8), (15, 5)])
    dims = [d for d in (64, 80, 96, 128, 192, 256) if heads * d != 3 * 1024]
    if op == "attn":
        dim = rng.choice(dims)
        batch, q_len = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5, 8, 16])
        # no more cache than the long listed case
        most = min(200000, 200000 * 8 * 128 // (kv_heads * dim * batch))
        if q_len > 1:
            most = min(most, 100000 // q_len)
        len_max = _log(rng, 16, max(17, most))
        window = rng.choice([0, 0, 0, _log(rng, 16, 8192)])
        return {"op": op, "type": kind, "batch": batch, "q_len": q_len, "heads": heads,
                "kv_heads": kv_heads, "head_dim": dim, "page": rng.choice([1, 16, 16, 24, 64, 256]),
                "len_min": rng.randint(1, len_max), "len_max": len_max, "window": window,
                "sinks": rng.choice([0, 4, 100]) if window else 0}
    if op == "append":
        dim = rng.choice(dims)
        len_max = _log(rng, 16, 2000)
        return {"op": op, "type": kind, "batch": _log(rng, 1, 128), "q_len": rng.choice([1, 2, 7, 16]),
                "heads": heads, "kv_heads": kv_heads, "head_dim": dim,
                "rot": rng.choice([dim, dim // 2, 16]), "page": rng.choice([1, 16, 24, 64]),
                "len_min": rng.randint(1, len_max), "len_max": len_max, "inter": rng.randint(0, 1)}
    if op == "norm":
        width = _log(rng, 100, 16384)
        return {"op": op, "type": kind, "rows": _log(rng, 1, max(2, 4096 * 4096 // width)), "width": width,
                "layer": rng.randint(0, 1), "post": rng.randint(0, 1), "gate": rng.randint(0, 2),
                "h32": rng.randint(0, 1)}
    int4 = rng.randint(0, 1)
    experts = rng.choice([8, 16, 33, 64, 128, 256])
    hidden = _log(rng, 8, 64, 64)
    # no more weights than the wide listed case
    inter = _log(rng, 4, min(224, 8 * 14336 * 4096 // (experts * hidden * 64)), 64)
    return {"op": "moe", "type": "f16" if int4 else kind, "int4": int4, "tokens": rng.randint(1, 16),
            "hidden": hidden, "inter": inter, "experts": experts,
            "top_k": rng.randint(1, 2 if experts < 33 else 8)}


# ---- inputs ---------------------------------------------------------------------------

def _lengths(c):
    """The sequences' lengths (new tokens included): spread from len_min to
    len_max over their logarithm; a property of the case."""
    n, lo, hi = c["batch"], c["len_min"], c["len_max"]
    if n == 1:
        return [hi]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** (i / (n - 1)))))) for i in range(n)]


def _visible(c, length):
    """Cache positions that some new token of a sequence sees."""
    first = max(0, length - c["q_len"])
    lo = max(0, first - c["window"] + 1) if c["window"] else 0
    return length - lo + min(lo, c["sinks"])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, dt = dict(case), _DTYPE[case["type"]]

    def normal(shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)

    s = {"case": c}
    if c["op"] in ("attn", "append"):
        lens = _lengths(c)
        random.Random(seed).shuffle(lens)
        B, page = c["batch"], c["page"]
        max_pages = -(-max(lens) // page) + 1
        used = [-(-n // page) for n in lens]
        num_pages = sum(used) + 3
        # a program's pages lie scattered over the pool; unused table entries are -1
        order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32).cpu()
        table, at = torch.full((B, max_pages), -1, dtype=torch.int32), 0
        for b in range(B):
            table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
        s["table"] = table.to(DEV)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        D, Hk = c["head_dim"], c["kv_heads"]
        s["k_cache"] = torch.empty(num_pages, page, Hk, D, dtype=dt, device=DEV)
        s["v_cache"] = torch.empty(num_pages, page, Hk, D, dtype=dt, device=DEV)
        for cache in (s["k_cache"], s["v_cache"]):
            cache.normal_(0.0, 1.0, generator=g)
        tokens = B * c["q_len"]
        if c["op"] == "attn":
            s["q"] = normal((tokens, c["heads"], D), 1.5)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(tokens, c["heads"], dtype=torch.float32, device=DEV)
        else:
            # q, k and v as one product's output row, as a fused q|k|v matrix leaves them
            width = (c["heads"] + 2 * Hk) * D
            qkv = normal((tokens, width))
            s["q"] = qkv[:, :c["heads"] * D].view(tokens, c["heads"], D)
            s["k"] = qkv[:, c["heads"] * D:(c["heads"] + Hk) * D].view(tokens, Hk, D)
            s["v"] = qkv[:, (c["heads"] + Hk) * D:].view(tokens, Hk, D)
            s["q_out"] = torch.empty(tokens, c["heads"], D, dtype=dt, device=DEV)
            half = c["rot"] // 2
            freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
            ang = torch.arange(c["len_max"], device=DEV, dtype=torch.float64)[:, None] * freq
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    elif c["op"] == "norm":
        M, N = c["rows"], c["width"]
        hdt = torch.float32 if c["h32"] else dt
        s["y"] = normal((M, N), 0.7)
        s["h"] = normal((M, N), 2.0, hdt)
        s["w_pre"] = (1.0 + 0.2 * torch.randn(N, generator=g, device=DEV)).to(dt)
        s["b_pre"] = normal((N,), 0.1) if c["layer"] else None
        s["w_post"] = (1.0 + 0.2 * torch.randn(N, generator=g, device=DEV)).to(dt) if c["post"] else None
        s["b_post"] = normal((N,), 0.1) if c["post"] and c["layer"] else None
        # gate 1: one factor for each value; 2: one row of factors for all tokens
        s["gate"] = normal((M, N) if c["gate"] == 1 else (N,), 0.5) if c["gate"] else None
        s["alpha"], s["beta"], s["eps"] = 1.0, 0.8, 1e-6
        s["h_out"], s["x_out"] = torch.empty_like(s["h"]), torch.empty(M, N, dtype=dt, device=DEV)
    else:
        M, K, I, E = c["tokens"], c["hidden"], c["inter"], c["experts"]
        s["x"] = normal((M, K))
        s["router"] = normal((E, K), 1.0 / math.sqrt(K))
        for name, n, k in (("gate", I, K), ("up", I, K), ("down", K, I)):
            if c["int4"]:  # codes -7..7 two to a byte, even k low; fp16 scale of each 32
                s["w_" + name] = torch.empty(E, n, k // 2, dtype=torch.uint8, device=DEV)
                for e in range(E):
                    q = torch.randint(-7, 8, (n, k), generator=g, device=DEV, dtype=torch.int8)
                    s["w_" + name][e] = ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).view(torch.uint8)
                u = torch.rand(E, n, k // 32, generator=g, device=DEV)
                s["s_" + name] = ((0.1 + u) / (2.5 * math.sqrt(k))).to(torch.float16)
            else:
                s["w_" + name] = torch.empty(E, n, k, dtype=dt, device=DEV)
                s["w_" + name].normal_(0.0, 1.0 / math.sqrt(k), generator=g)
                s["s_" + name] = None
        s["y"] = torch.empty(M, K, dtype=dt, device=DEV)
        s["ids"] = torch.empty(M, c["top_k"], dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(M, c["top_k"], dtype=torch.float32, device=DEV)
    if own:
        _describe(s)
    return s


def _describe(s):
    """The descriptors and workspace that a program keeps beside its buffers."""
    import quantized_skinny_gemm_gb300 as dg
    c, need = s["case"], 0
    if c["op"] in ("attn", "append"):
        kv = dg.paged_kv(s["k_cache"], s["v_cache"], s["table"], s["lens"])
        if c["op"] == "attn":
            s["desc"] = dg.attention(kv, s["q"], s["out"], lse=s["lse"], q_len=c["q_len"],
                                     window=c["window"], sinks=c["sinks"])
            need = dg.attn_workspace_bytes(s["desc"])
        else:
            s["desc"] = dg.append(kv, s["q"], s["k"], s["v"], s["q_out"], q_len=c["q_len"],
                                  cos=s["cos"], sin=s["sin"], interleaved=bool(c["inter"]))
    elif c["op"] == "norm":
        s["desc"] = dg.norm(s["h"], s["h_out"], s["x_out"], s["w_pre"], b_pre=s["b_pre"], y=s["y"],
                            w_post=s["w_post"], b_post=s["b_post"], gate=s["gate"],
                            alpha=s["alpha"], beta=s["beta"], eps=s["eps"],
                            kind=dg.NORM_LAYER if c["layer"] else dg.NORM_RMS)
    else:
        kind = dg.LINEAR_W4A16 if c["int4"] else dg.LINEAR_F16 if c["type"] == "f16" else dg.LINEAR_BF16
        s["desc"] = dg.moe(kind, s["x"], s["y"], s["router"], s["w_gate"], s["w_up"], s["w_down"],
                           c["top_k"], gate_scale=s["s_gate"], up_scale=s["s_up"],
                           down_scale=s["s_down"], ids=s["ids"], weights=s["weights"],
                           renormalize=True)
        need = dg.moe_workspace_bytes(s["desc"])
    s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None


# ---- one pass -------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import quantized_skinny_gemm_gb300 as dg
        if op == "attn":
            dg.attn_decode(s["desc"], s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "append":
            dg.kv_append(s["desc"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "norm":
            dg.norm_residual(s["desc"])
            return {"h": s["h_out"], "x": s["x_out"]}
        dg.moe_forward(s["desc"], s["ws"])
        return {"y": s["y"], "ids": s["ids"], "weights": s["weights"]}
    return {"attn": _attn, "append": _append, "norm": _norm, "moe": _moe}[op](s)


def _attn(s):
    c = s["case"]
    B, Q, Hk, D, page = c["batch"], c["q_len"], c["kv_heads"], c["head_dim"], c["page"]
    G = c["heads"] // Hk
    lens = s["lens"].long()
    first = (lens - Q).view(B, 1)
    span = s["table"].shape[1] * page
    if c["window"]:  # only the positions that some token can see
        lo = (first - c["window"] + 1).clamp(min=0)
        keep = c["sinks"] + c["window"] + Q - 1
        i = torch.arange(min(span, keep), device=DEV).view(1, -1)
        sinks = torch.minimum(lo, torch.full_like(lo, c["sinks"]))
        pos = torch.where(i < sinks, i, i - sinks + lo)
    else:
        pos = torch.arange(span, device=DEV).view(1, -1).expand(B, -1)
    pages = s["table"].gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1)).long()
    at = pages.clamp(min=0) * page + pos % page
    k = s["k_cache"].view(-1, Hk, D)[at].float()           # [B, L, Hk, D]
    q = s["q"].view(B, Q, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, Q * G, D).float()
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hk, Q, G, -1) / math.sqrt(D)
    del k
    p_q = (first + torch.arange(Q, device=DEV)).view(B, 1, Q, 1, 1)
    j = pos.view(B, 1, 1, 1, -1)
    seen = (j <= p_q) & (pages.view(B, 1, 1, 1, -1) >= 0)
    if c["window"]:
        seen &= (j > p_q - c["window"]) | (j < c["sinks"])
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(score - base)
    del score
    total = e.sum(-1, keepdim=True)
    v = s["v_cache"].view(-1, Hk, D)[at].float().permute(0, 2, 1, 3)
    out = torch.matmul(e.view(B, Hk, Q * G, -1), v).view(B, Hk, Q, G, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (base + torch.log(total)).squeeze(-1)
    heads = c["heads"]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B * Q, heads, D).to(s["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B * Q, heads)}


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    part, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        out = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        out = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((out, rest), -1)


def _append(s):
    c = s["case"]
    B, Q, page = c["batch"], c["q_len"], c["page"]
    pos = (s["lens"].long().view(B, 1) - Q + torch.arange(Q, device=DEV)).view(-1)
    live = pos >= 0
    row = pos.clamp(min=0)
    cos, sin = s["cos"][row], s["sin"][row]
    pages = s["table"].long().gather(1, (row // page).view(B, Q)).view(-1)
    q = _rotate(s["q"], cos, sin, c["rot"], c["inter"]) * live[:, None, None]
    k = _rotate(s["k"], cos, sin, c["rot"], c["inter"]).to(s["k"].dtype)
    # tokens before the sequence's start write nothing: they put back what is there
    first = live.view(B, Q).to(torch.int8).argmax(1)
    source = torch.maximum(torch.arange(Q, device=DEV).view(1, Q), first.view(B, 1))
    source = (source + torch.arange(B, device=DEV).view(B, 1) * Q).view(-1)
    page_at, slot = pages[source], (row % page)[source]
    s["k_cache"][page_at, slot] = k[source]
    s["v_cache"][page_at, slot] = s["v"][source]
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _normed(v, w, b, eps, layer):
    if layer:
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * w.float()
    return v + b.float() if b is not None else v


def _norm(s):
    r = s["y"].float()
    if s["w_post"] is not None:
        r = _normed(r, s["w_post"], s["b_post"], s["eps"], s["case"]["layer"])
    if s["gate"] is not None:
        r = r * s["gate"].float()
    h = s["alpha"] * s["h"].float() + s["beta"] * r
    x = _normed(h, s["w_pre"], s["b_pre"], s["eps"], s["case"]["layer"])
    return {"h": h.to(s["h"].dtype), "x": x.to(s["y"].dtype)}


def _weights_of(s, name, ids):
    """The chosen experts' matrices [tokens, top_k, rows, columns] in fp32."""
    w = s["w_" + name][ids]
    if not s["case"]["int4"]:
        return w.float()
    codes = torch.stack((w & 15, w >> 4), -1).flatten(-2).float()
    codes = codes - 16.0 * (codes > 7)
    scale = s["s_" + name][ids].float()
    return (codes.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def _moe(s):
    k = s["case"]["top_k"]
    x = s["x"].float()
    logits = torch.matmul(x, s["router"].float().t())
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    prob, order = torch.sort(e / e.sum(-1, keepdim=True), dim=-1, descending=True, stable=True)
    ids, weights = order[:, :k], prob[:, :k]
    weights = weights / weights.sum(-1, keepdim=True)
    xc = x[:, None, :, None]
    gate = torch.matmul(_weights_of(s, "gate", ids), xc)
    up = torch.matmul(_weights_of(s, "up", ids), xc)
    h = gate / (1.0 + torch.exp(-gate)) * up
    out = torch.matmul(_weights_of(s, "down", ids), h).squeeze(-1)
    y = (out * weights[..., None]).sum(1)
    return {"y": y.to(s["x"].dtype), "ids": ids.to(torch.int32), "weights": weights}


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "attn":
        tokens, D = c["batch"] * c["q_len"], c["head_dim"]
        seen = sum(_visible(c, n) for n in _lengths(c))
        row = 0  # (row, position) pairs of all new tokens
        for n in _lengths(c):
            for i in range(c["q_len"]):
                p = n - c["q_len"] + i
                if p >= 0:
                    lo = max(0, p - c["window"] + 1) if c["window"] else 0
                    row += p + 1 - lo + min(lo, c["sinks"])
        return {"bytes": seen * c["kv_heads"] * D * 4 + tokens * c["heads"] * (D * 4 + 4)
                + 4 * c["batch"] + 4 * sum(-(-_visible(c, n) // c["page"]) for n in _lengths(c)),
                "flops": 4.0 * row * c["heads"] * D}
    if c["op"] == "append":
        tokens = sum(min(c["q_len"], n) for n in _lengths(c))
        D = c["head_dim"]
        return {"bytes": tokens * ((c["heads"] + 2 * c["kv_heads"]) * D * 4 + c["rot"] * 4 + 4)
                + 4 * c["batch"],
                "flops": 3.0 * tokens * (c["heads"] + c["kv_heads"]) * c["rot"]}
    if c["op"] == "norm":
        M, N = c["rows"], c["width"]
        per = 2 + (8 if c["h32"] else 4) + 2 + (2 if c["gate"] == 1 else 0)
        one = 1 + c["layer"] + c["post"] * (1 + c["layer"]) + (1 if c["gate"] == 2 else 0)
        return {"bytes": M * N * per + 2 * N * one, "flops": 12.0 * M * N}
    M, K, I, E = c["tokens"], c["hidden"], c["inter"], c["experts"]
    distinct = E * (1.0 - (1.0 - c["top_k"] / E) ** M)   # expected, tokens choosing evenly
    per = 0.5 + 2.0 / 32 if c["int4"] else 2.0
    return {"bytes": distinct * 3 * I * K * per + E * K * 2 + M * K * 4 + 8 * M * c["top_k"],
            "flops": 6.0 * M * c["top_k"] * I * K + 2.0 * M * E * K}


# ---- the definitions in 64 bits ----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _attn64, "append": _append64, "norm": _norm64, "moe": _moe64}[case["op"]](s)


def _attn64(s):
    c = s["case"]
    Q, Hk, G, page = c["q_len"], c["kv_heads"], c["heads"] // c["kv_heads"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        for i in range(Q):
            p = n - Q + i
            if p < 0:
                continue
            pos = torch.arange(p + 1, device=DEV)
            if c["window"]:
                pos = pos[(pos > p - c["window"]) | (pos < c["sinks"])]
            where = s["table"][b].long()[pos // page]
            for h in range(Hk):
                k = s["k_cache"][where, pos % page, h].double()
                v = s["v_cache"][where, pos % page, h].double()
                q = s["q"][b * Q + i, h * G:(h + 1) * G].double()
                z = (q @ k.t()) / math.sqrt(c["head_dim"])
                top = z.max(dim=1).values
                e = torch.exp(z - top[:, None])
                out[b * Q + i, h * G:(h + 1) * G] = (e @ v) / e.sum(1)[:, None]
                lse[b * Q + i, h * G:(h + 1) * G] = top + e.sum(1).log()
    return {"out": out, "lse": lse}


def _append64(s):
    c = s["case"]
    Q, page, half = c["q_len"], c["page"], c["rot"] // 2
    lens = s["lens"].cpu().tolist()
    table = s["table"].cpu()
    if c["inter"]:
        one, two = torch.arange(half) * 2, torch.arange(half) * 2 + 1
    else:
        one, two = torch.arange(half), torch.arange(half) + half
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64)
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    q, k, v = (s[n].cpu().double() for n in ("q", "k", "v"))
    cos, sin = s["cos"].cpu().double(), s["sin"].cpu().double()
    where, new_k, new_v = [], [], []
    for t in range(q.shape[0]):
        p = lens[t // Q] - Q + t % Q
        if p < 0:
            continue
        turned = []
        for x in (q[t], k[t]):
            z = torch.complex(x[:, one], x[:, two]) * torch.complex(cos[p], sin[p])
            x = x.clone()
            x[:, one], x[:, two] = z.real, z.imag
            turned.append(x)
        q_out[t] = turned[0]
        where.append((int(table[t // Q, p // page]), p % page))
        new_k.append(turned[1])
        new_v.append(v[t])
    a = torch.tensor(where, device=DEV)
    caches[0][a[:, 0], a[:, 1]] = torch.stack(new_k).to(DEV)
    caches[1][a[:, 0], a[:, 1]] = torch.stack(new_v).to(DEV)
    return {"q": q_out, "k_cache": caches[0], "v_cache": caches[1]}


def _norm64(s):
    layer, eps = s["case"]["layer"], s["eps"]

    def f(v, w, b):
        if layer:
            d = v - v.sum(1, keepdim=True) / v.shape[1]
            y = d / torch.sqrt((d * d).sum(1, keepdim=True) / v.shape[1] + eps) * w.double()
            return y + b.double()
        return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + eps) * w.double()

    r = s["y"].double()
    r = f(r, s["w_post"], s["b_post"]) if s["w_post"] is not None else r
    r = r * s["gate"].double() if s["gate"] is not None else r
    h = s["alpha"] * s["h"].double() + s["beta"] * r
    return {"h": h, "x": f(h, s["w_pre"], s["b_pre"])}


def _moe64(s):
    c = s["case"]
    x = s["x"].double()
    z = x @ s["router"].double().t()
    prob = torch.softmax(z, 1)
    order = torch.argsort(prob, dim=1, descending=True, stable=True)[:, :c["top_k"]]
    weights = prob.gather(1, order)
    weights = weights / weights.sum(1, keepdim=True)
    y = torch.zeros(x.shape, dtype=torch.float64, device=DEV)

    def matrix(name, e):
        w = s["w_" + name][e]
        if not c["int4"]:
            return w.double()
        lut = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1],
                           dtype=torch.float64, device=DEV)
        full = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=DEV)
        full[:, 0::2], full[:, 1::2] = lut[(w & 15).long()], lut[(w >> 4).long()]
        return full * s["s_" + name][e].double().repeat_interleave(32, dim=1)

    for e in sorted(set(order.flatten().tolist())):
        tok, slot = torch.nonzero(order == e, as_tuple=True)
        xe = x[tok]
        a = xe @ matrix("gate", e).t()
        h = a * torch.sigmoid(a) * (xe @ matrix("up", e).t())
        y[tok] += weights[tok, slot][:, None] * (h @ matrix("down", e).t())
    return {"y": y, "ids": order.to(torch.int32), "weights": weights}
