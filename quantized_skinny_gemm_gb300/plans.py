"""Decode-step plans: a decoder's weights, inputs and outputs on the device,
marshalled once into the dg_linear array that dg_decode_step_weights runs.

The op order is the decoder's: per layer q, k, v (sharing x_attn), o, gate, up
(sharing x_mlp), down, then the lm_head.  The library fuses each run of ops
that share an input into one launch (q|k|v, gate|up).

Memory layout: weights (and scales) are separate, resident tensors, loaded
once; every activation a step reads lives in one input arena and every result
it writes in one output arena (256-byte aligned views), so moving a step's
inputs in and its results out is one copy each way.
"""
from dataclasses import dataclass, field
from typing import Dict, List, Optional

import torch

from . import (EPI_RESIDUAL, EPI_SWIGLU, LINEAR_F16, LINEAR_W4A16, LINEAR_W4A8, LINEAR_W8A8,
               StepPlan, append, attention, attn_decode, attn_workspace_bytes, decode_step_weights,
               kv_append, linear, moe, moe_forward, moe_workspace_bytes, norm, norm_residual,
               paged_kv, residual_add, swiglu)


class Arena:
    """One device buffer carved into aligned views: reserve(), then build()."""

    def __init__(self, align=256):
        self.align = align
        self.specs = []
        self.size = 0
        self.buf = None

    def reserve(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        off = self.size
        self.size = (off + nbytes + self.align - 1) // self.align * self.align
        self.specs.append((off, tuple(shape), dtype, nbytes))
        return len(self.specs) - 1

    def build(self, device):
        self.buf = torch.zeros(max(self.size, self.align), dtype=torch.uint8, device=device)
        return [self.buf[o:o + nb].view(dt).view(shape) for o, shape, dt, nb in self.specs]


@dataclass
class DeviceStep:
    plan: StepPlan
    ws: Optional[torch.Tensor]
    inputs: List[Dict[str, torch.Tensor]]      # per layer: name -> device fp16 [M][K]
    outputs: List[Dict[str, torch.Tensor]]     # per layer: matrix name -> device y [M][N]
    in_arena: torch.Tensor                     # every input of the step (uint8 bytes)
    out_arena: torch.Tensor                    # every result of the step (uint8 bytes)
    weight_bytes: int                          # weights + scales streamed per step
    n_launches: int                            # kernel launches per step
    head_logits: Optional[torch.Tensor] = None
    head_token: Optional[torch.Tensor] = None
    head_input: Optional[torch.Tensor] = None
    keep: list = field(default_factory=list)
    # W4A8: per layer, input name -> (int8 codes [M][K], fp32 scale [M]) that
    # the step writes when it quantizes that input (empty for W4A16)
    act_codes: List[Dict[str, tuple]] = field(default_factory=list)
    head_codes: Optional[tuple] = None


def _nbytes(t):
    return t.numel() * t.element_size()


def count_launches(ops, persistent=True):
    """Kernel launches (memsets excluded) dg_decode_step_weights issues for
    these ops: with the persistent kernel, one per run of single-token ops of
    one kind (per 144 fused groups); otherwise one per fused group (same kind,
    no epilogue,
    M, K, group and activation pointers, up to 4 ops, an lm_head alone), plus
    the lm_head's argmax pass and one quantization launch per fused group with
    fp16 inputs to an int8-activation kind."""
    def groups(lo, hi):
        out, i = [], lo
        while i < hi:
            a = ops[i]
            j = i + 1
            if not a.token and not a.epilogue:
                while j < hi and j - i < 4:
                    b = ops[j]
                    if (b.token or b.epilogue or b.kind != a.kind or b.M != a.M or b.K != a.K
                            or b.x != a.x
                            or b.x_i8 != a.x_i8 or b.x_scale != a.x_scale
                            or b.group_size != a.group_size):
                        break
                    j += 1
            out.append((i, j))
            i = j
        return out

    n, i = 0, 0
    while i < len(ops):
        j = i
        while persistent and j < len(ops) and ops[j].kind == ops[i].kind and ops[j].M == 1 \
                and not ops[j].acc_out:
            j += 1
        if j > i:
            g = len(groups(i, j))
            n += (g + 143) // 144
            i = j
            continue
        a, b = groups(i, len(ops))[0]
        op = ops[a]
        int8_act = op.kind in (LINEAR_W4A8, LINEAR_W8A8)
        n += 1 + (1 if op.token else 0) + (1 if int8_act and op.x else 0)
        i = b
    return n


def fp16_decode_step(layers, device, M=1) -> DeviceStep:
    """layers: synth.decode_fp16_workload(...) output (host tensors)."""
    ain, aout = Arena(), Arena()
    in_ids = [{k: ain.reserve(v.shape, torch.float16) for k, v in L.inputs.items()}
              for L in layers]
    out_ids = [{lin.name: aout.reserve((M, lin.N), torch.float16) for lin in L.linears}
               for L in layers]
    in_views, out_views = ain.build(device), aout.build(device)
    ops, keep, ins, outs = [], [], [], []
    wbytes = 0
    for L, iid, oid in zip(layers, in_ids, out_ids):
        xin = {}
        for k, v in L.inputs.items():
            xin[k] = in_views[iid[k]]
            xin[k].copy_(v)
        ys = {}
        for lin in L.linears:
            W = lin.W.to(device)
            y = out_views[oid[lin.name]]
            ops.append(linear(LINEAR_F16, W, M, lin.N, lin.K, x=xin[lin.x_name], y=y))
            keep.append(W)
            ys[lin.name] = y
            wbytes += _nbytes(W)
        ins.append(xin)
        outs.append(ys)
    keep += [ain.buf, aout.buf]
    plan = StepPlan(ops, keep)
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device=device)
    return DeviceStep(plan, ws, ins, outs, ain.buf, aout.buf, wbytes, count_launches(ops),
                      keep=keep)


def int4_decode_step(layers, head, x_head, device, act="a16", M=1, group=32) -> DeviceStep:
    """layers/head/x_head: synth.decode_int4_workload(...) output (host tensors).
    act="a16": fp16 activations; act="a8": per-token int8 activations, quantized
    inside the step from the fp16 inputs (scratch codes live in the workspace
    tensors kept by the plan)."""
    kind = LINEAR_W4A16 if act == "a16" else LINEAR_W4A8
    ain, aout = Arena(), Arena()
    in_ids = [{k: ain.reserve(v.shape, torch.float16) for k, v in L.inputs.items()}
              for L in layers]
    out_ids = [{lin.name: aout.reserve((M, lin.N), torch.float16) for lin in L.linears}
               for L in layers]
    head_ids = None
    if head is not None:
        head_ids = (ain.reserve(x_head.shape, torch.float16),
                    aout.reserve((head.N,), torch.float32), aout.reserve((1,), torch.int32))
    in_views, out_views = ain.build(device), aout.build(device)
    ops, keep, ins, outs = [], [], [], []
    codes = []
    wbytes = 0

    def qbufs(x):
        if act == "a16":
            return None, None
        xq = torch.empty(x.shape, dtype=torch.int8, device=device)
        xs = torch.empty(x.shape[0], dtype=torch.float32, device=device)
        keep.extend([xq, xs])
        return xq, xs

    for L, iid, oid in zip(layers, in_ids, out_ids):
        xin = {}
        for k, v in L.inputs.items():
            xin[k] = in_views[iid[k]]
            xin[k].copy_(v)
        qin = {k: qbufs(v) for k, v in xin.items()}
        codes.append({k: v for k, v in qin.items() if v[0] is not None})
        ys = {}
        for lin in L.linears:
            W, S = lin.W.to(device), lin.scales.to(device)
            y = out_views[oid[lin.name]]
            xq, xs = qin[lin.x_name]
            ops.append(linear(kind, W, M, lin.N, lin.K, w_scale=S, x=xin[lin.x_name], x_i8=xq,
                              x_scale=xs, y=y, group_size=group))
            keep += [W, S]
            ys[lin.name] = y
            wbytes += _nbytes(W) + _nbytes(S)
        ins.append(xin)
        outs.append(ys)
    logits = token = xh = None
    hcodes = None
    if head is not None and head.scales is None:
        # an fp16 lm_head after the int4 layers (a second persistent launch)
        W = head.W.to(device)
        xh = in_views[head_ids[0]]
        xh.copy_(x_head)
        logits, token = out_views[head_ids[1]], out_views[head_ids[2]]
        ops.append(linear(LINEAR_F16, W, 1, head.N, head.K, x=xh, logits=logits, token=token))
        keep.append(W)
        wbytes += _nbytes(W)
    elif head is not None:
        W, S = head.W.to(device), head.scales.to(device)
        xh = in_views[head_ids[0]]
        xh.copy_(x_head)
        logits, token = out_views[head_ids[1]], out_views[head_ids[2]]
        xq, xs = qbufs(xh)
        hcodes = (xq, xs) if xq is not None else None
        ops.append(linear(kind, W, 1, head.N, head.K, w_scale=S, x=xh, x_i8=xq, x_scale=xs,
                          logits=logits, token=token, group_size=group))
        keep += [W, S]
        wbytes += _nbytes(W) + _nbytes(S)
    keep += [ain.buf, aout.buf]
    plan = StepPlan(ops, keep)
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device=device)
    return DeviceStep(plan, ws, ins, outs, ain.buf, aout.buf, wbytes, count_launches(ops),
                      logits, token, xh, keep=keep, act_codes=codes, head_codes=hcodes)


@dataclass
class BlockStep:
    """A decoder-block step with its epilogues: fused (one dg_decode_step_weights
    call, residual and SwiGLU in the stream's epilogues) or unfused (the
    GEMVs, then separate elementwise launches).  run() enqueues one step."""
    run: object
    inputs: List[Dict[str, torch.Tensor]]      # per layer: x_attn, x_o, x_mlp, h
    outputs: List[Dict[str, torch.Tensor]]     # per layer: q, k, v, h1, act, h2
    in_arena: torch.Tensor
    out_arena: torch.Tensor
    weight_bytes: int
    n_launches: int
    plan: Optional[StepPlan] = None
    ws: Optional[torch.Tensor] = None
    keep: list = field(default_factory=list)


def fp16_block_step(layers, hs, device, fused=True) -> BlockStep:
    """The 1536-wide fp16 decoder as decoder blocks (synth.decode_fp16_workload
    layers, synth.residual_stream inputs hs).  Per layer: q, k, v = W x_attn;
    h1 = h + W_o x_o; act = silu(W_gate x_mlp) * (W_up x_mlp); h2 = h1 +
    W_down act.  The attention and the norms between them are not part of the
    weight stream: x_attn, x_o and x_mlp are synthetic inputs.  Fused: the
    residual adds and SwiGLU are epilogues of one persistent launch (down
    waits for act and h1 inside it).  Unfused: per layer the GEMVs of q, k, v,
    o, gate and up in one launch, then h1 = h + o, act = swiglu(gate, up),
    the down GEMV and h2 = h1 + down as launches of their own."""
    ain, aout = Arena(), Arena()
    M = 1
    names_in = ("x_attn", "x_o", "x_mlp")
    in_ids, out_ids = [], []
    for L, h in zip(layers, hs):
        hidden = h.shape[1]
        inter = next(l.N for l in L.linears if l.name == "gate")
        ids = {k: ain.reserve(L.inputs[k].shape, torch.float16) for k in names_in}
        ids["h"] = ain.reserve(h.shape, torch.float16)
        in_ids.append(ids)
        o = {n: aout.reserve((M, l.N), torch.float16) for l in L.linears for n in (l.name,)
             if n in ("q", "k", "v")}
        o["h1"] = aout.reserve((M, hidden), torch.float16)
        o["act"] = aout.reserve((M, inter), torch.float16)
        o["h2"] = aout.reserve((M, hidden), torch.float16)
        if not fused:  # the unfused GEMV outputs
            for n, width in (("o", hidden), ("gate", inter), ("up", inter), ("down", hidden)):
                o["y_" + n] = aout.reserve((M, width), torch.float16)
        out_ids.append(o)
    in_views, out_views = ain.build(device), aout.build(device)
    keep, ins, outs, wbytes = [ain.buf, aout.buf], [], [], 0
    fused_ops, per_layer = [], []
    for L, h, iid, oid in zip(layers, hs, in_ids, out_ids):
        xin = {k: in_views[iid[k]] for k in iid}
        for k in names_in:
            xin[k].copy_(L.inputs[k])
        xin["h"].copy_(h)
        ys = {k: out_views[oid[k]] for k in oid}
        W = {l.name: l.W.to(device) for l in L.linears}
        keep += list(W.values())
        wbytes += sum(_nbytes(w) for w in W.values())
        lin = {l.name: l for l in L.linears}
        mk = lambda n, x, y, **kw: linear(LINEAR_F16, W[n], M, lin[n].N, lin[n].K, x=x, y=y, **kw)
        qkv = [mk(n, xin["x_attn"], ys[n]) for n in ("q", "k", "v")]
        if fused:
            fused_ops += qkv + [
                mk("o", xin["x_o"], ys["h1"], epilogue=EPI_RESIDUAL, residual=xin["h"]),
                mk("gate", xin["x_mlp"], ys["act"], epilogue=EPI_SWIGLU, W2=W["up"]),
                mk("down", ys["act"], ys["h2"], epilogue=EPI_RESIDUAL, residual=ys["h1"])]
        else:
            head = qkv + [mk("o", xin["x_o"], ys["y_o"]), mk("gate", xin["x_mlp"], ys["y_gate"]),
                          mk("up", xin["x_mlp"], ys["y_up"])]
            down = [mk("down", ys["act"], ys["y_down"])]
            per_layer.append((StepPlan(head), StepPlan(down), xin, ys))
        ins.append(xin)
        outs.append(ys)
    if fused:
        plan = StepPlan(fused_ops, keep)
        ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device=device)
        run = lambda stream=None: decode_step_weights(plan, ws, stream=stream)
        return BlockStep(run, ins, outs, ain.buf, aout.buf, wbytes, 1, plan, ws, keep)
    wsb = max(max(a.workspace_bytes(), b.workspace_bytes()) for a, b, _, _ in per_layer)
    ws = torch.empty(wsb, dtype=torch.uint8, device=device)

    def run(stream=None):
        for head, down, xin, ys in per_layer:
            decode_step_weights(head, ws, stream=stream)
            residual_add(xin["h"], ys["y_o"], ys["h1"], stream=stream)
            swiglu(ys["y_gate"], ys["y_up"], ys["act"], stream=stream)
            decode_step_weights(down, ws, stream=stream)
            residual_add(ys["h1"], ys["y_down"], ys["h2"], stream=stream)
    keep.append(per_layer)
    return BlockStep(run, ins, outs, ain.buf, aout.buf, wbytes, 5 * len(per_layer), None, ws, keep)


@dataclass
class SparseStep:
    """A sparse decoder's whole step for the q_len new tokens of each sequence.
    run() enqueues one step: h in, h_out and x_out (normed) out, and the new
    tokens' keys and values into the caches.  Before each run seq_lens must
    count the new tokens and block_table must name the pages they fall in; both
    are read on the device, so a captured graph follows them."""
    run: object
    h: torch.Tensor                            # fp32 [batch * q_len][hidden]
    h_out: torch.Tensor                        # fp32
    x_out: torch.Tensor                        # fp16
    seq_lens: torch.Tensor                     # int32 [batch]
    block_table: torch.Tensor                  # int32 [batch][max_pages]
    caches: List[tuple]                        # per layer: k, v [pages][page_size][kv_heads][head_dim]
    layers: List[Dict[str, torch.Tensor]]      # per layer: q, k, v, q_rot, att, o, x, h_mid, x_mid, y, ids, weights
    keep: list = field(default_factory=list)


def sparse_decoder_step(layers, device, heads, kv_heads, top_k, final_norm=None, batch=1, q_len=1,
                        page_size=64, max_pages=16, window=0, sinks=0, group=32, rope=None,
                        share=None) -> SparseStep:
    """layers: synth.sparse_decoder_workload(...) output; batch * q_len from 1 to
    16; rope: (cos, sin) fp32 [max_pos][rot / 2] or None; share: another
    SparseStep of the same layers and batch (with another q_len) whose weights,
    tables, caches and lengths this one uses.  Per layer
      h += y (of the layer before); x = norm_attn(h); q, k, v = W x;
      rotate q and k, k and v into the cache; att = attention; o = W_o att;
      h += o; x = norm_mlp(h); y = experts(x)
    and last h += y; x_out = final_norm(h).  The residual stream stays fp32; the
    adds are part of the norms."""
    M, f16, f32, i32 = batch * q_len, torch.float16, torch.float32, torch.int32
    if batch < 1 or q_len < 1 or M > 16:
        raise ValueError("batch * q_len: the products and the experts take 1 to 16 rows")
    if share is not None and share.block_table.shape[0] != batch:
        raise ValueError("share: another batch")
    hidden = layers[0].q.shape[1]
    dim = layers[0].q.shape[0] // heads
    for L in layers:
        if any(tuple(w.shape) != (rows, cols) for w, rows, cols in (
                (L.q, heads * dim, hidden), (L.k, kv_heads * dim, hidden), (L.v, kv_heads * dim, hidden),
                (L.o, hidden, heads * dim))):
            raise ValueError("heads, kv_heads: the layers' q, k, v, o have other sizes")
    new = lambda *shape, dtype=f16: torch.zeros(shape, dtype=dtype, device=device)
    if share is None:
        pages = batch * max_pages
        lens = new(batch, dtype=i32)
        table = torch.arange(pages, dtype=i32, device=device).view(batch, max_pages)
        weights = [{k: v.to(device) for k, v in vars(L).items() if torch.is_tensor(v)} for L in layers]
        scales = [{k: v.to(device) for k, v in L.scales.items()} for L in layers]
        caches = [(new(pages, page_size, kv_heads, dim), new(pages, page_size, kv_heads, dim)) for _ in layers]
        final = (torch.ones(hidden, dtype=f16) if final_norm is None else final_norm).to(device)
        cos, sin = (None, None) if rope is None else (t.to(device) for t in rope)
    else:
        lens, table, caches = share.seq_lens, share.block_table, share.caches
        weights, scales, final, cos, sin = share.keep[0]
    first = h = new(M, hidden, dtype=f32)
    y, ops, views, attn_ws, moe_ws, lin_ws = None, [], [], 0, 0, 0
    for W, S, (kc, vc) in zip(weights, scales, caches):
        kv = paged_kv(kc, vc, table, lens)
        t = {"x": new(M, hidden), "q": new(M, heads * dim), "k": new(M, kv_heads * dim), "v": new(M, kv_heads * dim),
             "q_rot": new(M, heads * dim), "att": new(M, heads * dim), "o": new(M, hidden),
             "h": new(M, hidden, dtype=f32), "h_mid": new(M, hidden, dtype=f32), "x_mid": new(M, hidden),
             "y": new(M, hidden), "ids": new(M, top_k, dtype=i32), "weights": new(M, top_k, dtype=f32)}
        lin = lambda w, a, b: linear(LINEAR_F16, W[w], M, b.shape[1], a.shape[1], x=a, y=b)
        qkv = StepPlan([lin(n, t["x"], t[n]) for n in ("q", "k", "v")])
        out = StepPlan([lin("o", t["att"], t["o"])])
        att = attention(kv, t["q_rot"], t["att"], q_len=q_len, window=window, sinks=sinks)
        kind = LINEAR_W4A16 if S else LINEAR_F16
        experts = moe(kind, t["x_mid"], t["y"], W["router"], W["gate"], W["up"], W["down"], top_k,
                      gate_scale=S.get("gate"), up_scale=S.get("up"), down_scale=S.get("down"), ids=t["ids"],
                      weights=t["weights"], group_size=group, renormalize=True)
        ops.append((norm(h, t["h"], t["x"], W["norm_attn"], y=y), qkv,
                    append(kv, t["q"], t["k"], t["v"], q_out=t["q_rot"], q_len=q_len, cos=cos, sin=sin), att, out,
                    norm(t["h"], t["h_mid"], t["x_mid"], W["norm_mlp"], y=t["o"]), experts))
        if not attn_workspace_bytes(att):
            raise ValueError("the attention refuses these heads, window or strides")
        if not moe_workspace_bytes(experts):
            raise ValueError("the expert layer refuses these sizes")
        attn_ws = max(attn_ws, attn_workspace_bytes(att))
        moe_ws = max(moe_ws, moe_workspace_bytes(experts))
        lin_ws = max(lin_ws, qkv.workspace_bytes(), out.workspace_bytes())
        h, y = t["h_mid"], t["y"]
        views.append(t)
    h_out, x_out = new(M, hidden, dtype=f32), new(M, hidden)
    last = norm(h, h_out, x_out, final, y=y)
    ws_a, ws_m, ws_l = (new(max(n, 16), dtype=torch.uint8) for n in (attn_ws, moe_ws, lin_ws))

    def run(stream=None):
        for pre, qkv, app, att, out, mid, experts in ops:
            norm_residual(pre, stream=stream)
            decode_step_weights(qkv, ws_l, stream=stream)
            kv_append(app, stream=stream)
            attn_decode(att, ws_a, stream=stream)
            decode_step_weights(out, ws_l, stream=stream)
            norm_residual(mid, stream=stream)
            moe_forward(experts, ws_m, stream=stream)
        norm_residual(last, stream=stream)
    return SparseStep(run, first, h_out, x_out, lens, table, caches, views,
                      [(weights, scales, final, cos, sin), ws_a, ws_m, ws_l, share])
