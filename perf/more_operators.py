"""What a serving step runs around a 4-bit cache and its answer, as measured cases.

Four operators: pages and slots for the tokens to come (``pages``), head norms
and rotary positions with the append to a 16-bit or 4-bit paged cache
(``append``), attention of new tokens over the 4-bit cache (``attn4``), and log
probabilities of given tokens with entropy and alternatives (``logprobs``).
With ``own`` false, ``run`` computes them in plain 32-bit torch; with ``own``
true it calls the library's entry points.  ``exact`` evaluates the definitions
in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's first tokens: one sequence, a short cache, the 4096-wide decoder's heads
        {"name": "attn4 one short f16", "op": "attn4", "type": "f16", "batch": 1, "q_len": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "len_min": 100, "len_max": 100,
         "window": 0, "sinks": 0, "slot_major": 0},
        # a serving batch of ragged lengths on the 1536-wide decoder's heads
        {"name": "attn4 ragged batch bf16", "op": "attn4", "type": "bf16", "batch": 16, "q_len": 1,
         "heads": 12, "kv_heads": 2, "head_dim": 128, "page": 16, "len_min": 1, "len_max": 8191,
         "window": 0, "sinks": 0, "slot_major": 0},
        # one long document: the cache is the whole cost
        {"name": "attn4 one long bf16", "op": "attn4", "type": "bf16", "batch": 1, "q_len": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "len_min": 200001,
         "len_max": 200001, "window": 0, "sinks": 0, "slot_major": 0},
        # draft tokens verified under a sliding window with sink tokens, small heads
        {"name": "attn4 verify window f16", "op": "attn4", "type": "f16", "batch": 8, "q_len": 8,
         "heads": 32, "kv_heads": 8, "head_dim": 64, "page": 16, "len_min": 1500,
         "len_max": 40000, "window": 4096, "sinks": 4, "slot_major": 1},
        # one new token of one sequence into a 16-bit cache, heads of the 1536-wide decoder
        {"name": "append one f16", "op": "append", "type": "f16", "bits": 16, "batch": 1, "q_len": 1,
         "heads": 12, "kv_heads": 2, "head_dim": 128, "rot": 128, "page": 16, "len_min": 1000,
         "len_max": 1000, "inter": 0, "layer": 0, "map": 0},
        # draft tokens of a serving batch into a 4-bit cache, part of each head rotates, in pairs
        {"name": "append batch 4 bits bf16", "op": "append", "type": "bf16", "bits": 4, "batch": 256,
         "q_len": 8, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 64, "page": 16,
         "len_min": 17, "len_max": 700, "inter": 1, "layer": 0, "map": 0},
        # prompts of ragged lengths in one call, by their slots, layer norms of the heads
        {"name": "append prompts 4 bits f16", "op": "append", "type": "f16", "bits": 4, "batch": 13,
         "q_len": 0, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128, "page": 64,
         "len_min": 33, "len_max": 2000, "inter": 0, "layer": 1, "map": 1},
        # a decode step of a serving batch: a page now and then
        {"name": "pages decode step", "op": "pages", "batch": 64, "page": 16, "len_max": 4000,
         "new_max": 1, "ended": 0, "short": 0},
        # prompts join and sequences end, and the pool runs out
        {"name": "pages prompts join", "op": "pages", "batch": 3000, "page": 16, "len_max": 8000,
         "new_max": 700, "ended": 5, "short": 1},
        # the alternatives of one decoded token, the 4096-wide decoder's vocabulary
        {"name": "logprobs one f32", "op": "logprobs", "type": "f32", "rows": 1, "vocab": 128256,
         "top_k": 5, "scale": 1.25},
        # draft tokens of a batch, a wide vocabulary, with masked words
        {"name": "logprobs verify f32", "op": "logprobs", "type": "f32", "rows": 61, "vocab": 248320,
         "top_k": 20, "scale": 1.0},
        # scoring a prompt, an odd vocabulary
        {"name": "logprobs scoring bf16", "op": "logprobs", "type": "bf16", "rows": 2047,
         "vocab": 128255, "top_k": 1, "scale": 1.0},
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn4", "attn4", "attn4", "append", "append", "pages", "logprobs", "logprobs"])
    kind = rng.choice(["f16", "bf16"])
    heads, kv_heads = rng.choice([(12, 2), (32, 8), (16, 16), (28, 4), (20, 1), (40, 8), (15, 5)])
    dim = rng.choice([64, 80, 96, 128, 192, 256])
    page = rng.choice([1, 16, 16, 24, 64, 256])
    if op == "attn4":
        batch, q_len = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5, 8, 16])
        # no more cache than the long listed case
        most = min(200000, 200000 * 8 * 128 // (kv_heads * dim * batch))
        if q_len > 1:
            most = min(most, 100000 // q_len)
        len_max = _log(rng, 16, max(17, most))
        window = rng.choice([0, 0, 0, _log(rng, 16, 8192)])
        return {"op": op, "type": kind, "batch": batch, "q_len": q_len, "heads": heads,
                "kv_heads": kv_heads, "head_dim": dim, "page": page,
                "len_min": rng.randint(1, len_max), "len_max": len_max, "window": window,
                "sinks": rng.choice([0, 4, 100]) if window else 0, "slot_major": rng.randint(0, 1)}
    if op == "append":
        bits, by_map = rng.choice([4, 16]), rng.randint(0, 1)
        batch = _log(rng, 1, 16 if by_map else 128)
        len_max = _log(rng, 16, 1000 if by_map else 2000)
        return {"op": op, "type": kind, "bits": bits, "batch": batch,
                "q_len": 0 if by_map else rng.choice([1, 2, 7, 16]), "heads": heads,
                "kv_heads": kv_heads, "head_dim": dim, "rot": rng.choice([dim, dim // 2, 16, 0]),
                "page": page, "len_min": rng.randint(1, len_max), "len_max": len_max,
                "inter": rng.randint(0, 1), "layer": rng.randint(0, 1), "map": by_map}
    if op == "pages":
        return {"op": op, "batch": _log(rng, 1, 3000), "page": page, "len_max": _log(rng, 16, 8000),
                "new_max": rng.choice([1, 1, 8, 16, _log(rng, 16, 700)]),
                "ended": rng.choice([0, 3, 20]), "short": rng.randint(0, 1)}
    vocab = _log(rng, 1000, 250000)
    kind = rng.choice(["f16", "bf16", "f32", "f32"])
    rows = _log(rng, 1, max(2, 2047 * 128255 // (vocab * (2 if kind == "f32" else 1))))
    return {"op": op, "type": kind, "rows": rows, "vocab": vocab,
            "top_k": rng.choice([0, 1, 5, 20, 32]), "scale": rng.choice([1.0, 0.5, 1.25])}


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
    c, s = dict(case), {"case": dict(case)}

    def normal(shape, std=1.0, dtype=None):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std
        return x.to(_DTYPE[c["type"]] if dtype is None else dtype)

    def randint(lo, hi, shape, dtype=torch.int32):
        return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=dtype)

    if c["op"] in ("attn4", "append"):
        _prepare_cache(s, seed, g, normal, randint)
    elif c["op"] == "pages":
        B, P = c["batch"], c["page"]
        s["lens"] = (torch.rand(B, generator=g, device=DEV) ** 2 * c["len_max"]).to(torch.int32)
        s["new"] = randint(1, c["new_max"] + 1, (B,))
        # some sequences join (nothing held yet), some end
        s["lens"] = torch.where(torch.rand(B, generator=g, device=DEV) < 0.2,
                                torch.zeros_like(s["lens"]), s["lens"])
        if c["ended"]:
            gone = torch.rand(B, generator=g, device=DEV) * 100 < c["ended"]
            s["new"] = torch.where(gone, torch.full_like(s["new"], -1), s["new"])
        held = (s["lens"] + P - 1) // P
        wide = (c["len_max"] + c["new_max"] + P - 1) // P
        used, most = int(held.sum()), B * wide
        order = torch.randperm(most, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((B, wide), -1, dtype=torch.int32, device=DEV)
        at = torch.cumsum(held, 0) - held
        col = torch.arange(wide, device=DEV).view(1, -1)
        s["table"] = torch.where(col < held.view(-1, 1),
                                 order[(at.view(-1, 1) + col).clamp(max=most - 1)], s["table"])
        # a pool that was in use for a while: its queue begins anywhere
        want = s["new"].clamp(min=0)
        need = int((((s["lens"] + want + P - 1) // P) - held).sum())
        free = max(1, need * 2 // 3) if c["short"] else most - used
        first = int(randint(0, most, (1,)))
        s["pool"] = torch.full((most,), -1, dtype=torch.int32, device=DEV)
        s["pool"][(torch.arange(free, device=DEV) + first) % most] = order[used:used + free]
        s["pool_state"] = torch.tensor([first, free], dtype=torch.int32, device=DEV)
        tokens = B * c["new_max"]   # the program's buffers for a step
        s["lens_out"], s["state_out"] = torch.empty_like(s["lens"]), torch.empty_like(s["pool_state"])
        s["starts"] = torch.empty(B + 1, dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(tokens, dtype=torch.int64, device=DEV)
        s["positions"] = torch.empty(tokens, dtype=torch.int32, device=DEV)
    else:
        R, V = c["rows"], c["vocab"]
        s["logits"] = torch.empty(R, V, dtype=_DTYPE[c["type"]], device=DEV)
        s["logits"].normal_(0.0, 2.5, generator=g)
        if c["rows"] > 1 and c["type"] == "f32":   # words that the program has ruled out
            s["logits"][:, randint(0, V, (V // 50,), torch.int64)] = -math.inf
        # tokens as a sampler takes them: mostly likely ones
        u = torch.rand(R, 1, generator=g, device=DEV).clamp(min=1e-6)
        some = randint(0, V, (R, 64), torch.int64)
        best = s["logits"].gather(1, some).float().argmax(1, keepdim=True)
        s["tokens"] = torch.where(u < 0.7, some.gather(1, best), some[:, :1]).to(torch.int32).view(R)
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=DEV)
        s["logprob"], s["entropy"], s["lse"] = new(R), new(R), new(R)
        s["rank"] = new(R, dtype=torch.int32)
        s["top_ids"], s["top_logprobs"] = new(R, c["top_k"], dtype=torch.int32), new(R, c["top_k"])
    if own:
        _describe(s)
    return s


def _prepare_cache(s, seed, g, normal, randint):
    c = s["case"]
    dt = _DTYPE[c["type"]]
    lens = _lengths(c)
    random.Random(seed).shuffle(lens)
    B, P, D, Hk = c["batch"], c["page"], c["head_dim"], c["kv_heads"]
    max_pages = -(-max(lens) // P) + 1
    used = [-(-n // P) for n in lens]
    num_pages = sum(used) + 3
    # a program's pages lie scattered over the pool; unused table entries are -1
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32).cpu()
    table, at = torch.full((B, max_pages), -1, dtype=torch.int32), 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    s["table"] = table.to(DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    bits = 4 if c["op"] == "attn4" else c["bits"]
    s["cache"] = {}
    for n in ("k", "v"):
        if bits == 16:
            s["cache"][n] = torch.empty(num_pages, P, Hk, D, dtype=dt, device=DEV)
            s["cache"][n].normal_(0.0, 1.0, generator=g)
            continue
        # [page][head][slot] in memory, or [page][slot][head]; always seen as [page][slot][head]
        lie = (num_pages, P, Hk) if c.get("slot_major") else (num_pages, Hk, P)
        view = (lambda t: t) if c.get("slot_major") else (lambda t: t.transpose(1, 2))
        s["cache"][n] = view(randint(0, 256, lie + (D // 2,), torch.uint8))
        # scales near 0.3, as values of unit size have them (e4m3: 0.25 to 0.47)
        s["cache"][n + "_scale"] = view(randint(0x28, 0x30, lie + (D // 16,), torch.uint8))
    s["k_factor"], s["v_factor"] = 0.75, 1.5
    if c["op"] == "attn4":
        tokens = B * c["q_len"]
        s["q"] = normal((tokens, c["heads"], D), 1.5)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(tokens, c["heads"], dtype=torch.float32, device=DEV)
        return
    if c["map"]:   # every token of the sequences, in order
        pos = np.concatenate([np.arange(n) for n in lens])
        seq = np.repeat(np.arange(B), lens)
        s["positions"] = torch.from_numpy(pos).to(torch.int32).to(DEV)
        s["slots"] = (table.numpy()[seq, pos // P].astype(np.int64) * P + pos % P)
        s["slots"] = torch.from_numpy(s["slots"]).to(DEV)
        tokens = len(pos)
    else:
        tokens = B * c["q_len"]
    # q, k and v as one product's output row, as a fused q|k|v matrix leaves them
    qkv = normal((tokens, (c["heads"] + 2 * Hk) * D))
    s["q"] = qkv[:, :c["heads"] * D].view(tokens, c["heads"], D)
    s["k"] = qkv[:, c["heads"] * D:(c["heads"] + Hk) * D].view(tokens, Hk, D)
    s["v"] = qkv[:, (c["heads"] + Hk) * D:].view(tokens, Hk, D)
    s["q_out"] = torch.empty(tokens, c["heads"], D, dtype=dt, device=DEV)
    s["w_q"], s["w_k"] = (1.0 + normal((D,), 0.2, torch.float32)).to(dt), (1.0 + normal((D,), 0.2, torch.float32)).to(dt)
    s["eps"] = 1e-6
    half = c["rot"] // 2
    s["cos"] = s["sin"] = None
    if half:
        freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        ang = torch.arange(c["len_max"], device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    if bits == 4:
        s["k_read"], s["v_read"] = (torch.empty(tokens, Hk, D, dtype=dt, device=DEV) for _ in "kv")


def _describe(s):
    """The descriptors and workspace that a program keeps beside its buffers."""
    import quantized_skinny_gemm_gb300 as dg
    c, need = s["case"], 0
    if c["op"] in ("attn4", "append"):
        h = s["cache"]
        if "k_scale" in h:
            kv = dg.paged_kv4(h["k"], h["v"], h["k_scale"], h["v_scale"], s["table"], s["lens"],
                              dtype=_DTYPE[c["type"]], k_factor=s["k_factor"], v_factor=s["v_factor"])
        else:
            kv = dg.paged_kv(h["k"], h["v"], s["table"], s["lens"])
        if c["op"] == "attn4":
            s["desc"] = dg.attention4(kv, s["q"], s["out"], lse=s["lse"], q_len=c["q_len"],
                                      window=c["window"], sinks=c["sinks"])
            need = dg.attn4_workspace_bytes(s["desc"])
        else:
            where = ({"slots": s["slots"], "positions": s["positions"]} if c["map"] else
                     {"q_len": c["q_len"]})
            s["desc"] = dg.head_append(kv, s["q"], s["k"], s["v"], s["q_out"], cos=s["cos"],
                                       sin=s["sin"], interleaved=bool(c["inter"]), w_q=s["w_q"],
                                       w_k=s["w_k"], eps=s["eps"],
                                       kind=dg.NORM_LAYER if c["layer"] else dg.NORM_RMS, **where)
            if c["bits"] == 4:
                where.pop("positions", None)
                s["read"] = dg.kv4_rows(kv, s["k_read"], s["v_read"], **where)
    elif c["op"] == "pages":
        s["desc"] = dg.page_plan(s["lens"], s["table"], s["pool"], s["pool_state"], c["page"],
                                 new_lens=s["new"], lens_out=s["lens_out"],
                                 pool_state_out=s["state_out"], starts=s["starts"],
                                 slots=s["slots"], positions=s["positions"])
        need = dg.pages_workspace_bytes(s["desc"])
    else:
        k = c["top_k"]
        s["desc"] = dg.logprobs(s["logits"], tokens=s["tokens"], logprob=s["logprob"],
                                rank=s["rank"], entropy=s["entropy"], lse=s["lse"],
                                top_ids=s["top_ids"] if k else None,
                                top_logprobs=s["top_logprobs"] if k else None, scale=c["scale"])
        need = dg.logprobs_workspace_bytes(s["desc"])
    s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None


# ---- one pass -------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        import quantized_skinny_gemm_gb300 as dg
        if op == "attn4":
            dg.attn4_decode(s["desc"], s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "append":
            dg.qkv_append(s["desc"])
            if "read" not in s:
                return {"q": s["q_out"], "k": s["cache"]["k"], "v": s["cache"]["v"]}
            dg.kv4_read(s["read"])   # what now lies in the tokens' places
            return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
        if op == "pages":
            dg.assign_pages(s["desc"], s["ws"])
            return {"lens": s["lens_out"], "table": s["table"], "pool": s["pool"],
                    "state": s["state_out"], "starts": s["starts"], "slots": s["slots"],
                    "positions": s["positions"]}
        dg.token_logprobs(s["desc"], s["ws"])
        return {n: s[n] for n in ("logprob", "rank", "entropy", "lse", "top_ids", "top_logprobs")}
    return {"attn4": _attn4, "append": _append, "pages": _pages, "logprobs": _logprobs}[op](s)


def _e4m3(byte):
    """Values of e4m3 bytes in fp32."""
    b = byte.to(torch.int32)
    e, m = (b >> 3) & 15, b & 7
    v = torch.where(e > 0, torch.ldexp((8 + m).float(), e - 10), m.float() * 2.0 ** -9)
    v = torch.where((e == 15) & (m == 7), torch.full_like(v, math.nan), v)
    return torch.where(b > 127, -v, v)


def _decoded(codes, scales, factor):
    """codes [..., D / 2] and scales [..., D / 16] -> values [..., D] in fp32."""
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int8)
    x = torch.where(x > 7, x - 16, x).float().unflatten(-1, (-1, 16))
    return (x * (_e4m3(scales) * factor)[..., None]).flatten(-2)


def _coded(x, factor):
    """values [..., D] in fp32 -> codes, scales."""
    g = x.unflatten(-1, (-1, 16))
    top = g.abs().amax(-1, keepdim=True)
    byte = (top / (7.0 * factor)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = byte.float() * factor
    q = torch.where(step > 0, torch.round(g / torch.where(step > 0, step, torch.ones_like(step))),
                    torch.zeros_like(g)).clamp(-7, 7).to(torch.int32).flatten(-2) & 15
    return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8), byte.squeeze(-1).view(torch.uint8)


def _attn4(s):
    c, h = s["case"], s["cache"]
    B, Q, Hk, D, P = c["batch"], c["q_len"], c["kv_heads"], c["head_dim"], c["page"]
    G = c["heads"] // Hk
    first = (s["lens"].long() - Q).view(B, 1)
    span = s["table"].shape[1] * P
    if c["window"]:  # only the positions that some token can see
        lo = (first - c["window"] + 1).clamp(min=0)
        keep = c["sinks"] + c["window"] + Q - 1
        i = torch.arange(min(span, keep), device=DEV).view(1, -1)
        sinks = torch.minimum(lo, torch.full_like(lo, c["sinks"]))
        pos = torch.where(i < sinks, i, i - sinks + lo)
    else:
        pos = torch.arange(span, device=DEV).view(1, -1).expand(B, -1)
    pages = s["table"].gather(1, (pos // P).clamp(max=s["table"].shape[1] - 1)).long()
    page, slot = pages.clamp(min=0), pos % P
    k = _decoded(h["k"][page, slot], h["k_scale"][page, slot], s["k_factor"])   # [B, L, Hk, D]
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
    v = _decoded(h["v"][page, slot], h["v_scale"][page, slot], s["v_factor"]).permute(0, 2, 1, 3)
    out = torch.matmul(e.view(B, Hk, Q * G, -1), v).view(B, Hk, Q, G, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (base + torch.log(total)).squeeze(-1)
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B * Q, c["heads"], D).to(s["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B * Q, c["heads"])}


def _head_normed(x, w, eps, layer):
    x = x.float()
    if layer:
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _rotate(x, cos, sin, rot, interleaved):
    if not rot:
        return x
    part, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        out = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        out = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((out, rest), -1)


def _places(s):
    """Position, page and slot of each of the append's tokens; position < 0: none."""
    c = s["case"]
    B, Q, P = c["batch"], c["q_len"], c["page"]
    if c["map"]:
        return s["positions"].long(), s["slots"] // P, s["slots"] % P
    pos = (s["lens"].long().view(B, 1) - Q + torch.arange(Q, device=DEV)).view(-1)
    row = pos.clamp(min=0)
    return pos, s["table"].long().gather(1, (row // P).view(B, Q)).view(-1), row % P


def _append(s):
    c, h, dt = s["case"], s["cache"], s["q"].dtype
    pos, page, slot = _places(s)
    live = pos >= 0
    row = pos.clamp(min=0)
    cos, sin = (s["cos"][row], s["sin"][row]) if c["rot"] else (None, None)
    q = _rotate(_head_normed(s["q"], s["w_q"], s["eps"], c["layer"]), cos, sin, c["rot"], c["inter"])
    k = _rotate(_head_normed(s["k"], s["w_k"], s["eps"], c["layer"]), cos, sin, c["rot"], c["inter"])
    q = (q * live[:, None, None]).to(dt)
    # tokens before the sequence's start write nothing: they put back what the first one writes
    source = torch.arange(len(pos), device=DEV)
    if not c["map"]:
        B, Q = c["batch"], c["q_len"]
        first = live.view(B, Q).to(torch.int8).argmax(1)
        source = torch.maximum(torch.arange(Q, device=DEV).view(1, Q), first.view(B, 1))
        source = (source + torch.arange(B, device=DEV).view(B, 1) * Q).view(-1)
    at = (page[source], slot[source])
    if c["bits"] == 16:
        h["k"][at] = k[source].to(dt)
        h["v"][at] = s["v"][source]
        return {"q": q, "k": h["k"], "v": h["v"]}
    read = []
    for n, x, f in (("k", k, s["k_factor"]), ("v", s["v"].float(), s["v_factor"])):
        codes, scales = _coded(x[source], f)
        h[n][at], h[n + "_scale"][at] = codes, scales
        read.append((_decoded(h[n][page, slot], h[n + "_scale"][page, slot], f)
                     * live[:, None, None]).to(dt))
    return {"q": q, "k": read[0], "v": read[1]}


def _pages(s):
    c = s["case"]
    P, N, T = c["page"], s["pool"].numel(), s["slots"].numel()
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"]
    first, count = s["pool_state"].long()
    ended, want = new < 0, new.clamp(min=0)
    held, total = (lens + P - 1) // P, lens + want
    need = (total + P - 1) // P
    ends = torch.cumsum(want, 0)
    starts = torch.cat((torch.zeros_like(ends[:1]), ends))
    fits = ~ended & (need <= table.shape[1]) & (ends <= T)
    more = torch.where(fits, need - held, torch.zeros_like(need))
    upto = torch.cumsum(more, 0)
    served = fits & ((more == 0) | (upto <= count))
    col = torch.arange(table.shape[1], device=DEV).view(1, -1)
    grown = served.view(-1, 1) & (col >= held.view(-1, 1)) & (col < need.view(-1, 1))
    number = (upto - more - held).view(-1, 1) + col
    rows = torch.where(grown, s["pool"][(first + number.clamp(min=0)) % N], table)
    taken = torch.where(served & (more > 0), upto, torch.zeros_like(upto)).amax()
    back = torch.where(ended, held, torch.zeros_like(held))
    given = torch.cumsum(back, 0)
    gives = col < back.view(-1, 1)
    at = ((given - back).view(-1, 1) + col + first + count) % N
    pool = s["pool"].clone()
    pool[at[gives]] = table[gives]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(ends, t, right=True)
    inside = seq < lens.numel()
    seq = seq.clamp(max=lens.numel() - 1)
    pos = lens[seq] + t - starts[seq]
    ok = inside & served[seq]
    slot = rows[seq, (pos // P).clamp(max=table.shape[1] - 1)].long() * P + pos % P
    none = torch.full_like(t, -1)
    zero = torch.zeros_like(lens)
    return {"lens": torch.where(ended, zero, torch.where(served, total, lens)).to(torch.int32),
            "table": rows, "pool": pool,
            "state": torch.stack(((first + taken) % N, count - taken + back.sum())).to(torch.int32),
            "starts": starts.to(torch.int32), "slots": torch.where(ok, slot, none),
            "positions": torch.where(ok, pos, none).to(torch.int32)}


def _logprobs(s):
    c = s["case"]
    raw = s["logits"].float()
    z = raw * c["scale"]
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    below = (z - top).clamp(min=-1e30)
    entropy = (torch.log(total) - (e * below).sum(-1, keepdim=True) / total).view(-1)
    del e, below, z
    token = s["tokens"].long().view(-1, 1)
    mine = raw.gather(1, token)
    word = torch.arange(raw.shape[1], device=DEV).view(1, -1)
    rank = ((raw > mine) | ((raw == mine) & (word < token))).sum(-1)
    best, order = torch.sort(raw, dim=-1, descending=True, stable=True)
    k = c["top_k"]
    return {"logprob": (mine * c["scale"] - lse).view(-1), "rank": rank.to(torch.int32),
            "entropy": entropy, "lse": lse.view(-1), "top_ids": order[:, :k].to(torch.int32),
            "top_logprobs": best[:, :k] * c["scale"] - lse}


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "attn4":
        tokens, D = c["batch"] * c["q_len"], c["head_dim"]
        seen = sum(_visible(c, n) for n in _lengths(c))
        pairs = 0  # (row, position) pairs of all new tokens
        for n in _lengths(c):
            for p in range(max(0, n - c["q_len"]), n):
                lo = max(0, p - c["window"] + 1) if c["window"] else 0
                pairs += p + 1 - lo + min(lo, c["sinks"])
        return {"bytes": seen * c["kv_heads"] * (D + D // 8) + tokens * c["heads"] * (D * 4 + 4)
                + 4 * c["batch"] + 4 * sum(-(-_visible(c, n) // c["page"]) for n in _lengths(c)),
                "flops": 4.0 * pairs * c["heads"] * D}
    if c["op"] == "append":
        D, heads, kv = c["head_dim"], c["heads"], c["kv_heads"]
        tokens = sum(n if c["map"] else min(c["q_len"], n) for n in _lengths(c))
        stored = 2 * kv * (2 * D if c["bits"] == 16 else D // 2 + D // 16)
        read = 2 * kv * D * 2 if c["bits"] == 4 else 0   # what the cache gives back
        return {"bytes": tokens * ((2 * heads + 2 * kv) * D * 2 + stored + read + c["rot"] * 4
                                   + (12 if c["map"] else 4)) + 4 * c["batch"] + 4 * D,
                "flops": tokens * (heads + kv) * (6.0 * D + 3.0 * c["rot"]) + tokens * kv * 4.0 * D}
    if c["op"] == "pages":
        B = c["batch"]
        tokens = B * c["new_max"]
        grown = (B * (c["new_max"] + 1) / 2) / c["page"] * (2 / 3 if c["short"] else 1)
        back = B * c["ended"] / 100 * c["len_max"] / 3 / c["page"]
        return {"bytes": 16 * B + 12 * tokens + 8 * (grown + back), "flops": 20.0 * B + 4.0 * tokens}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * (4 if c["type"] == "f32" else 2) + c["rows"] * (20 + 8 * c["top_k"]),
            "flops": 8.0 * n}


# ---- the definitions in 64 bits ----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn4": _attn64, "append": _append64, "pages": _pages64,
            "logprobs": _logprobs64}[case["op"]](s)


def _tables64():
    """Values of the 16 codes and of the 256 scale bytes."""
    code = [i if i < 8 else i - 16 for i in range(16)]
    scale = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if b & 127 == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        scale.append(-v if b > 127 else v)
    return (torch.tensor(code, dtype=torch.float64, device=DEV),
            torch.tensor(scale, dtype=torch.float64, device=DEV))


def _stored64(codes, scales, factor):
    code, scale = _tables64()
    x = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.float64, device=DEV)
    x[..., 0::2], x[..., 1::2] = code[(codes & 15).long()], code[(codes >> 4).long()]
    return x * scale[scales.long()].repeat_interleave(16, dim=-1) * factor


def _attn64(s):
    c, h = s["case"], s["cache"]
    Q, G, P = c["q_len"], c["heads"] // c["kv_heads"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        every = torch.arange(n, device=DEV)
        if c["window"]:
            every = every[(every > n - Q - c["window"]) | (every < c["sinks"])]
        where, slot = s["table"][b].long()[every // P], every % P
        for g in range(c["kv_heads"]):
            k = _stored64(h["k"][where, slot, g], h["k_scale"][where, slot, g], s["k_factor"])
            v = _stored64(h["v"][where, slot, g], h["v_scale"][where, slot, g], s["v_factor"])
            for i in range(max(0, Q - n), Q):
                p = n - Q + i
                see = every <= p
                if c["window"]:
                    see &= (every > p - c["window"]) | (every < c["sinks"])
                q = s["q"][b * Q + i, g * G:(g + 1) * G].double()
                z = (q @ k[see].t()) / math.sqrt(c["head_dim"])
                top = z.max(dim=1).values
                e = torch.exp(z - top[:, None])
                out[b * Q + i, g * G:(g + 1) * G] = (e @ v[see]) / e.sum(1)[:, None]
                lse[b * Q + i, g * G:(g + 1) * G] = top + e.sum(1).log()
    return {"out": out, "lse": lse}


def _append64(s):
    c, h = s["case"], s["cache"]
    half, eps = c["rot"] // 2, s["eps"]
    pos, page, slot = _places(s)
    live = pos >= 0
    one = torch.arange(half, device=DEV) * (2 if c["inter"] else 1)
    two = one + (1 if c["inter"] else half)

    def turned(x, w):
        x = x.double()
        if c["layer"]:
            x = x - x.sum(-1, keepdim=True) / x.shape[-1]
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * w.double()
        if half:
            at = pos.clamp(min=0)
            z = torch.complex(x[..., one], x[..., two])
            z = z * torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
            x[..., one], x[..., two] = z.real, z.imag
        return x

    q, k, v = turned(s["q"], s["w_q"]), turned(s["k"], s["w_k"]), s["v"].double()
    q[~live] = 0.0
    if c["bits"] == 16:
        caches = [h["k"].double(), h["v"].double()]
        for cache, x in zip(caches, (k, v)):
            cache[page[live], slot[live]] = x[live]
        return {"q": q, "k": caches[0], "v": caches[1]}
    scales = _tables64()[1][:127]
    read = []
    for x, f in ((k, s["k_factor"]), (v, s["v_factor"])):
        g = x.unflatten(-1, (-1, 16)) / f
        want = (g.abs().amax(-1) / 7).clamp(max=448.0)
        hi = torch.searchsorted(scales, want).clamp(max=126)   # the first scale that is not below
        lo = (hi - 1).clamp(min=0)
        up, down = scales[hi] - want, want - scales[lo]
        pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        step = scales[pick][..., None]
        code = torch.where(step > 0, torch.round(g / torch.where(step > 0, step, 1.0)), 0.0).clamp(-7, 7)
        y = (code * step * f).flatten(-2)
        y[~live] = 0.0
        read.append(y)
    return {"q": q, "k": read[0], "v": read[1]}


def _pages64(s):
    """One sequence after the other, on the host."""
    c = s["case"]
    P = c["page"]
    lens, new, table, pool = (s[n].cpu().numpy().copy() for n in ("lens", "new", "table", "pool"))
    first, count = (int(x) for x in s["pool_state"].tolist())
    N, T = len(pool), s["slots"].numel()
    slots, positions = np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    starts, taken, asked, given, tail = [0], 0, 0, 0, first + count
    for b in range(len(lens)):
        n, w = int(lens[b]), int(new[b])
        held = -(-n // P)
        starts.append(starts[-1] + max(w, 0))
        if w < 0:
            pool[(tail + given + np.arange(held)) % N] = table[b, :held]
            given += held
            lens[b] = 0
            continue
        need = -(-(n + w) // P)
        if need > table.shape[1] or starts[-1] > T:
            continue
        asked += need - held
        if need > held:
            if asked > count:
                continue
            table[b, held:need] = pool[(first + taken + np.arange(need - held)) % N]
            taken = asked
        lens[b] = n + w
        p = n + np.arange(w)
        slots[starts[-2]:starts[-1]] = table[b, p // P].astype(np.int64) * P + p % P
        positions[starts[-2]:starts[-1]] = p
    state = np.array([(first + taken) % N, count - taken + given], np.int32)
    return {"lens": lens, "table": table, "pool": pool, "state": state,
            "starts": np.array(starts, np.int32), "slots": slots, "positions": positions}


def _logprobs64(s):
    c = s["case"]
    k, parts = c["top_k"], []
    for r in range(0, c["rows"], 256):   # some rows at a time
        z = s["logits"][r:r + 256].double() * c["scale"]
        lse = torch.logsumexp(z, -1, keepdim=True)
        lp = z - lse
        entropy = -torch.where(lp == -math.inf, 0.0, lp.exp() * lp).sum(-1)
        mine = lp.gather(1, s["tokens"][r:r + 256].long().view(-1, 1)).view(-1)
        parts.append((mine, entropy, lse.view(-1), lp.topk(k, dim=-1).values))
    mine, entropy, lse, best = (torch.cat(p) for p in zip(*parts))
    return {"logprob": mine, "rank": None, "entropy": entropy, "lse": lse, "top_ids": None,
            "top_logprobs": best}
