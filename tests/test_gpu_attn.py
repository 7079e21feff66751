"""Attention over the paged cache (dg_attn_decode) and the rotary append
(dg_kv_append) against the definitions in 64 bits: head layouts, head sizes,
page sizes, lengths around tiles, windows with sinks, tokens that see nothing,
NaN and infinity where nothing may see them, strides and layouts, far offsets,
streams and graphs."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _pool(lens, page, heads, dim, dt, seed, spare=2, garbage=None):
    """Host caches with scattered pages, table with -1 past each length;
    slots that hold no position get `garbage`."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    k = torch.randn(pages, page, heads, dim, generator=g)
    v = torch.randn(pages, page, heads, dim, generator=g)
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(max(used), 1) + 1), -1, dtype=torch.int32)
    held = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, :used[b]] = order[at:at + used[b]].int()
        for j in range(n):
            held[order[at + j // page], j % page] = True
        at += used[b]
    if garbage is not None:
        k[~held] = garbage
        v[~held] = garbage
    return k.to(dt), v.to(dt), table


def _run(k, v, table, lens, q, ftype, q_len=1, window=0, sinks=0, scale=None):
    kd, vd, td = k.to(DEV), v.to(DEV), table.to(DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qd = q.to(DEV)
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV)
    kv = dg.paged_kv(kd, vd, td, ld)
    op = dg.attention(kv, qd, out, lse=lse, q_len=q_len, window=window, sinks=sinks, scale=scale)
    ws = torch.full((dg.attn_workspace_bytes(op),), 255, dtype=torch.uint8, device=DEV)
    dg.attn_decode(op, ws)
    sync()
    return out, lse


def _check(k, v, table, lens, q, ftype, q_len=1, window=0, sinks=0, scale=None, what=""):
    out, lse = _run(k, v, table, lens, q, ftype, q_len, window, sinks, scale)
    s = q.shape[2] ** -0.5 if scale is None else scale
    ro, rl, bo, bl = ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), table.numpy(), lens, q_len, s,
                                   window, sinks, ftype)
    ref.check(ref.f64(out), ro, bo, what + " out")
    ref.check(ref.f64(lse), rl, bl, what + " lse")
    return out, lse


def _q(tokens, heads, dim, dt, seed, std=1.5):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(tokens, heads, dim, generator=g) * std).to(dt)


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("ftype,heads,kv_heads,dim,page,q_len,window,sinks", [
    ("f16", 4, 4, 64, 16, 1, 0, 0),
    ("f16", 32, 8, 128, 16, 1, 0, 0),
    ("bf16", 12, 2, 128, 64, 1, 0, 0),
    ("bf16", 6, 1, 256, 1, 1, 0, 0),
    ("f16", 15, 5, 80, 24, 1, 0, 0),
    ("f16", 3, 1, 8, 5, 1, 0, 0),
    ("bf16", 20, 1, 72, 16, 1, 0, 0),
    ("f16", 2, 2, 192, 256, 1, 0, 0),
    ("f16", 33, 1, 96, 16, 1, 0, 0),
    ("bf16", 8, 2, 64, 16, 2, 0, 0),
    ("f16", 12, 2, 128, 16, 5, 0, 0),
    ("f16", 32, 8, 128, 64, 16, 0, 0),
    ("bf16", 7, 1, 256, 24, 16, 0, 0),
    ("f16", 4, 4, 64, 16, 1, 1, 0),
    ("f16", 4, 2, 64, 16, 1, 16, 4),
    ("bf16", 12, 2, 128, 16, 1, 100, 1),
    ("bf16", 4, 4, 64, 3, 8, 33, 4),
    ("f16", 12, 2, 128, 16, 16, 64, 70),
    ("f16", 5, 5, 40, 7, 3, 1, 2),
    ("f16", 8, 1, 128, 16, 4, 5, 0),
])
def test_layouts_lengths_and_windows(ftype, heads, kv_heads, dim, page, q_len, window, sinks):
    need_gpu()
    dt = DT[ftype]
    k, v, table = _pool(LENS, page, kv_heads, dim, dt, 3)
    q = _q(len(LENS) * q_len, heads, dim, dt, 4)
    _check(k, v, table, LENS, q, ftype, q_len, window, sinks, what="attn")


@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ftype,q_len,window,sinks", [("f16", 1, 0, 0), ("bf16", 1, 40, 4),
                                                      ("f16", 4, 0, 0), ("bf16", 5, 40, 4)])
def test_what_a_token_does_not_see_never_reaches_it(ftype, q_len, window, sinks, garbage):
    """Unwritten slots, later draft tokens and positions that left the window
    hold NaN or infinities; only rows that do see one may show it."""
    need_gpu()
    lens, dim, page, dt = [3, 70, 129, 300], 64, 16, DT[ftype]
    k, v, table = _pool(lens, page, 2, dim, dt, 5, garbage=garbage)
    for b, n in enumerate(lens):
        for j in {n - 1, max(0, n - q_len + 1)}:      # seen by some rows of the step, not by all
            for c in (k, v):
                c[table[b, j // page], j % page, 1] = garbage
        if window and n > window + q_len + sinks:     # left the window for every row, or some
            for j in (sinks, n - window - q_len, n - window - 1):
                v[table[b, j // page], j % page] = garbage
                k[table[b, j // page], j % page] = garbage
    q = _q(len(lens) * q_len, 6, dim, dt, 6)
    out, _ = _run(k, v, table, lens, q, ftype, q_len, window, sinks)
    ro, _, bo, _ = ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), table.numpy(), lens, q_len,
                                 dim ** -0.5, window, sinks, ftype)
    fine = np.isfinite(ro).all(-1)
    assert fine.any()
    got = ref.f64(out)
    assert not np.isfinite(got[~fine]).all(-1).any()
    ref.check(got[fine], ro[fine], bo[fine], "rows that see finite values")


@pytest.mark.parametrize("q_len", [1, 6])
def test_missing_pages_are_unseen(q_len):
    need_gpu()
    lens, dim, page = [100, 64, 33], 128, 16
    k, v, table = _pool(lens, page, 2, dim, torch.float16, 7)
    table[0, 2] = -1
    table[0, 5] = k.shape[0]          # past the pool
    table[1, :] = -1                  # no page at all
    table[2, 1] = -7
    q = _q(3 * q_len, 8, dim, torch.float16, 8)
    out, lse = _check(k, v, table, lens, q, "f16", q_len, what="holes")
    assert (out[q_len:2 * q_len] == 0).all() and (lse[q_len:2 * q_len] == -float("inf")).all()


def test_length_past_the_table_stops_at_the_table():
    need_gpu()
    k, v, table = _pool([64], 16, 1, 64, torch.float16, 9)
    table = table[:, :4].contiguous()
    q = _q(1, 4, 64, torch.float16, 9)
    _check(k, v, table, [1000], q, "f16", what="clamped")
    _check(k, v, table, [2 ** 31 - 1], q, "f16", what="largest length")
    _check(k, v, table, [-5], q, "f16", what="negative length")


def test_scores_of_minus_infinity_and_nan():
    """All visible scores -inf: 0 and -inf.  A visible NaN key: NaN rows."""
    need_gpu()
    k, v, table = _pool([40, 40, 40], 16, 1, 64, torch.float16, 10)
    q = _q(3, 2, 64, torch.float16, 11).abs()
    for j in range(40):
        k[table[0, j // 16], j % 16] = -float("inf")
    k[table[1, 1], 3, 0, 5] = float("nan")
    k[table[2, 1], 3] = -float("inf")              # one token out of forty
    out, lse = _check(k, v, table, [40, 40, 40], q, "f16", what="inf / nan scores")
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()


@pytest.mark.parametrize("scale", [0.0, 4.0, -0.3])
def test_large_zero_and_negative_scales(scale):
    need_gpu()
    lens = [1, 200, 513]
    k, v, table = _pool(lens, 16, 2, 128, torch.bfloat16, 12)
    q = _q(3, 8, 128, torch.bfloat16, 13)
    _check(k, v, table, lens, q, "bf16", scale=scale, what="scale %g" % scale)


def test_values_of_the_types_range():
    """Scores near the fp32 range's useful end and values near fp16's."""
    need_gpu()
    lens = [150]
    k, v, table = _pool(lens, 16, 1, 64, torch.float16, 14)
    q = _q(1, 4, 64, torch.float16, 14, std=200.0)
    _check(k, (v * 15000).to(torch.float16), table, lens, q, "f16", what="large")


@pytest.mark.parametrize("ftype,heads,kv_heads,dim,lens", [
    ("bf16", 32, 8, 128, [20011]),
    ("f16", 12, 2, 128, [9001, 3, 511, 0, 4096]),
    ("f16", 16, 1, 64, [30000, 1]),
])
def test_long_and_ragged_caches(ftype, heads, kv_heads, dim, lens):
    need_gpu()
    k, v, table = _pool(lens, 16, kv_heads, dim, DT[ftype], 15)
    q = _q(len(lens), heads, dim, DT[ftype], 16)
    _check(k, v, table, lens, q, ftype, what="long")


def test_many_sequences():
    need_gpu()
    lens = [(i * 37) % 130 for i in range(700)]
    k, v, table = _pool(lens, 16, 1, 64, torch.float16, 17)
    q = _q(700, 2, 64, torch.float16, 18)
    _check(k, v, table, lens, q, "f16", what="700 sequences")


def test_layouts_strides_and_repeatability():
    """A [page][head][slot][dim] cache, both halves of one pool tensor, q and
    out as columns of wider rows, a table with its own stride; the same bits on
    another stream and on every call, with any workspace contents."""
    need_gpu()
    lens, heads, G, dim, page, q_len = [2500, 40, 700], 12, 2, 128, 16, 2
    k, v, table = _pool(lens, page, G, dim, torch.float16, 19)
    q = _q(len(lens) * q_len, heads, dim, torch.float16, 20)
    base, base_lse = _check(k, v, table, lens, q, "f16", q_len, what="plain layout")
    pool = torch.stack((k, v), 1).permute(0, 1, 3, 2, 4).contiguous().to(DEV)   # [P][2][G][S][D]
    kd, vd = pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2)
    wide = torch.full((len(lens) * q_len, heads * dim + 64), 7.0, dtype=torch.float16, device=DEV)
    wide[:, :heads * dim] = q.reshape(-1, heads * dim).to(DEV)
    outw = torch.full_like(wide, 9.0)
    tw = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    tw[:, :table.shape[1]] = table.to(DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    view = lambda w: w.as_strided((len(lens) * q_len, heads, dim), (w.shape[1], dim, 1))
    lse = torch.empty(len(lens) * q_len, heads, dtype=torch.float32, device=DEV)
    op = dg.attention(dg.paged_kv(kd, vd, tw[:, :table.shape[1]], ld), view(wide), view(outw), lse=lse,
                      q_len=q_len)
    sync()
    s = torch.cuda.Stream()
    for fill in (0, 255, 127):
        ws = torch.full((dg.attn_workspace_bytes(op),), fill, dtype=torch.uint8, device=DEV)
        outw.fill_(9.0)
        s.wait_stream(torch.cuda.current_stream())
        dg.attn_decode(op, ws, stream=s)
        s.synchronize()
        assert torch.equal(view(outw), base) and torch.equal(lse, base_lse)
        assert (outw[:, heads * dim:] == 9.0).all()


def test_offsets_past_32_bits():
    """A pool whose pages lie more than 2^32 bytes (2^31 elements) apart."""
    need_gpu()
    dim, page, stride = 64, 16, 1 << 27
    buf = torch.empty(2, 18 * stride, dtype=torch.float16, device=DEV)   # 2 x 4.8 GB
    g = torch.Generator().manual_seed(21)
    small = torch.randn(2, 18, page, 1, dim, generator=g).half()
    caches = [b.as_strided((18, page, 1, dim), (stride, dim, dim, 1)) for b in buf]
    for c, sm in zip(caches, small):
        c.copy_(sm.to(DEV))
    lens = [17 * page + 3]
    table = torch.tensor([[17, 3, 16, 0, 2, 15, 1, 4, 14, 5, 13, 6, 12, 7, 11, 8, 10, 9]],
                         dtype=torch.int32)
    q = _q(1, 4, dim, torch.float16, 22)
    out = torch.empty(1, 4, dim, dtype=torch.float16, device=DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    td, qd = table.to(DEV), q.to(DEV)
    kv = dg.paged_kv(*caches, td, ld)
    op = dg.attention(kv, qd, out)
    ws = torch.empty(dg.attn_workspace_bytes(op), dtype=torch.uint8, device=DEV)
    dg.attn_decode(op, ws)
    sync()
    ro, _, bo, _ = ref.attention(ref.f64(q), ref.f64(small[0]), ref.f64(small[1]), table.numpy(), lens, 1,
                                 dim ** -0.5)
    ref.check(ref.f64(out), ro, bo, "far pages")
    # and the append into the far page
    knew, vnew = _q(1, 1, dim, torch.float16, 23).to(DEV), _q(1, 1, dim, torch.float16, 24).to(DEV)
    dg.kv_append(dg.append(kv, None, knew, vnew))
    sync()
    where = int(table[0, (lens[0] - 1) // page]), (lens[0] - 1) % page
    assert torch.equal(caches[0][where], knew[0]) and torch.equal(caches[1][where], vnew[0])


def test_a_captured_step_follows_the_lengths():
    """append + attention captured once, replayed while the lengths grow."""
    need_gpu()
    heads, G, dim, page, steps = 8, 2, 64, 16, 20
    k, v, table = _pool([40], page, G, dim, torch.float16, 25)
    kd, vd, td = k.to(DEV), v.to(DEV), table.to(DEV)
    ld = torch.tensor([30], dtype=torch.int32, device=DEV)
    qkv = torch.empty(1, (heads + 2 * G) * dim, dtype=torch.float16, device=DEV)
    part = lambda a, n: qkv[:, a * dim:(a + n) * dim].view(1, n, dim)
    q, kn, vn = part(0, heads), part(heads, G), part(heads + G, G)
    ang = torch.arange(64).double()[:, None] * 10000.0 ** (-torch.arange(dim // 2).double() / (dim // 2))
    cos, sin = ang.cos().float(), ang.sin().float()
    cd, sd = cos.to(DEV), sin.to(DEV)
    q_out, out = torch.empty(1, heads, dim, dtype=torch.float16, device=DEV), \
        torch.empty(1, heads, dim, dtype=torch.float16, device=DEV)
    kv = dg.paged_kv(kd, vd, td, ld)
    ap = dg.append(kv, q, kn, vn, q_out, cos=cd, sin=sd)
    at = dg.attention(kv, q_out, out)
    ws = torch.empty(dg.attn_workspace_bytes(at), dtype=torch.uint8, device=DEV)
    dg.kv_append(ap)
    dg.attn_decode(at, ws)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ld.add_(1)
        dg.kv_append(ap)
        dg.attn_decode(at, ws)
    ld.fill_(30)
    kd.copy_(k.to(DEV))
    vd.copy_(v.to(DEV))
    kh, vh = ref.f64(k), ref.f64(v)
    for step in range(steps // 2):
        n = 31 + step
        row = _q(1, heads + 2 * G, dim, torch.float16, 100 + step)
        qkv.copy_(row.view(1, -1).to(DEV))
        graph.replay()
        sync()
        r = ref.f64(row)
        rq, kh, vh, bq, bk = ref.append(r[:, :heads], r[:, heads:heads + G], r[:, heads + G:], kh, vh,
                                        table.numpy(), [n], 1, ref.f64(cos), ref.f64(sin), False, "f16")
        ref.check(ref.f64(q_out), rq, bq, "rotated q, step %d" % step)
        ref.check(ref.f64(kd), kh, bk + 1e-12, "keys, step %d" % step)
        assert np.array_equal(ref.f64(vd), vh)
        kh, vh = ref.f64(kd), ref.f64(vd)              # go on from what the device holds
        ro, _, bo, _ = ref.attention(ref.f64(q_out), kh, vh, table.numpy(), [n], 1, dim ** -0.5)
        ref.check(ref.f64(out), ro, bo, "attention, step %d" % step)


# ---- the append -------------------------------------------------------------------------

@pytest.mark.parametrize("ftype,heads,kv_heads,dim,rot,inter,page,q_len", [
    ("f16", 12, 2, 128, 128, 0, 16, 1),
    ("bf16", 32, 8, 128, 64, 1, 16, 8),
    ("f16", 4, 4, 64, 0, 0, 16, 3),
    ("bf16", 5, 1, 72, 20, 0, 7, 2),
    ("f16", 3, 3, 80, 80, 1, 1, 16),
    ("f16", 2, 1, 8, 2, 1, 5, 4),
    ("bf16", 16, 2, 256, 256, 0, 64, 1),
    ("f16", 0, 2, 96, 48, 0, 16, 2),
])
def test_append(ftype, heads, kv_heads, dim, rot, inter, page, q_len):
    need_gpu()
    dt, lens = DT[ftype], [0, 1, 5, 16, 17, 40, 33, 39]
    k_cache, v_cache, table = _pool(lens, page, kv_heads, dim, dt, 30)
    table[5, 35 // page] = -1                 # a hole where tokens of sequence 5 would go
    T = len(lens) * q_len
    x = _q(T, heads + 2 * kv_heads, dim, dt, 31)
    q, kn, vn = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    half, max_pos = rot // 2, 38              # positions 38 and 39 are past the table
    ang = torch.arange(max_pos).double()[:, None] * 10000.0 ** (-torch.arange(half).double() / max(half, 1))
    cos, sin = (ang.cos().float(), ang.sin().float()) if rot else (None, None)
    on = lambda t: None if t is None else t.to(DEV)
    kd, vd, td = on(k_cache), on(v_cache), on(table)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qd, q_out = (on(q.contiguous()), torch.full((T, heads, dim), 5.0, dtype=dt, device=DEV)) if heads \
        else (None, None)
    kv = dg.paged_kv(kd, vd, td, ld)
    xd = x.to(DEV)                            # k and v as columns of one tensor
    kc = xd.view(T, -1)[:, heads * dim:].as_strided((T, kv_heads, dim), (xd.stride(0), dim, 1),
                                                    heads * dim)
    vc = xd.as_strided((T, kv_heads, dim), (xd.stride(0), dim, 1), (heads + kv_heads) * dim)
    cd, sd = on(cos), on(sin)
    dg.kv_append(dg.append(kv, qd, kc, vc, q_out, q_len=q_len, cos=cd, sin=sd, interleaved=bool(inter)))
    sync()
    rq, rk, rv, bq, bk = ref.append(ref.f64(q), ref.f64(kn), ref.f64(vn), ref.f64(k_cache),
                                    ref.f64(v_cache), table.numpy(), lens, q_len,
                                    None if cos is None else ref.f64(cos),
                                    None if sin is None else ref.f64(sin), inter, ftype)
    if heads:
        ref.check(ref.f64(q_out), rq, bq, "q")
        dg.kv_append(dg.append(kv, qd, kc, vc, q_len=q_len, cos=cd, sin=sd, interleaved=bool(inter)))
        sync()
        assert torch.equal(qd, q_out)         # in place
    ref.check(ref.f64(kd), rk, bk, "k cache")
    assert np.array_equal(ref.f64(vd), rv)


def test_append_at_any_alignment():
    """Pointers and strides that 16-byte vectors cannot take."""
    need_gpu()
    dim, heads, G, lens = 64, 3, 1, [9, 20]
    k_cache, v_cache, table = _pool(lens, 16, G, dim, torch.float16, 33)
    x = _q(2, heads + 2 * G, dim, torch.float16, 34)
    buf = torch.zeros(2 * 5 * dim + 64, dtype=torch.float16, device=DEV)
    xd = buf[3:3 + 2 * 5 * dim].view(2, 5, dim)
    xd.copy_(x.to(DEV))
    ang = torch.arange(32).double()[:, None] * 10000.0 ** (-torch.arange(32).double() / 32)
    cos, sin = ang.cos().float(), ang.sin().float()
    kd, vd, td = k_cache.to(DEV), v_cache.to(DEV), table.to(DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q_out = torch.empty(2, heads, dim, dtype=torch.float16, device=DEV)
    cd, sd = cos.to(DEV), sin.to(DEV)
    sub = lambda a, n: buf.as_strided((2, n, dim), (5 * dim, dim, 1), 3 + a * dim)
    dg.kv_append(dg.append(dg.paged_kv(kd, vd, td, ld), sub(0, 3), sub(3, 1), sub(4, 1), q_out,
                           cos=cd, sin=sd))
    sync()
    r = ref.f64(x)
    rq, rk, rv, bq, bk = ref.append(r[:, :3], r[:, 3:4], r[:, 4:], ref.f64(k_cache), ref.f64(v_cache),
                                    table.numpy(), lens, 1, ref.f64(cos), ref.f64(sin), False, "f16")
    ref.check(ref.f64(q_out), rq, bq, "q")
    ref.check(ref.f64(kd), rk, bk, "k")
    assert np.array_equal(ref.f64(vd), rv)
