"""Attention over the 4-bit cache (dg_attn4_decode) against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
import serve_ref
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 300]


def pool(lens, page, heads, dim, seed, spare=2, junk=None, lo=0x20, hi=0x38):
    """codes and scales [pages][page][heads][..] on the host, scattered pages, -1 past each
    length; slots that hold no position get scales of `junk`."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    u8 = lambda w, a, b: torch.randint(a, b, (pages, page, heads, w), generator=g, dtype=torch.uint8)
    cache = {"k": u8(dim // 2, 0, 256), "v": u8(dim // 2, 0, 256), "ks": u8(dim // 16, lo, hi),
             "vs": u8(dim // 16, lo, hi)}
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(max(used), 1) + 1), -1, dtype=torch.int32)
    held, at = torch.zeros(pages, page, dtype=torch.bool), 0
    for b, n in enumerate(lens):
        table[b, :used[b]] = order[at:at + used[b]].int()
        for j in range(n):
            held[order[at + j // page], j % page] = True
        at += used[b]
    if junk is not None:
        cache["ks"][~held] = junk
        cache["vs"][~held] = junk
    return cache, table


def lay(t, head_major):
    """On the device, [page][head][slot] in memory or [page][slot][head]."""
    return t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if head_major else t.contiguous().to(DEV)


def query(tokens, heads, dim, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(tokens, heads, dim, generator=g) * std).to(dt)


def run(cache, table, lens, q, q_len=1, window=0, sinks=0, scale=None, kf=1.0, vf=1.0, head_major=True, ws=None):
    d = {n: lay(t, head_major) for n, t in cache.items()}
    td, ld, qd = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), q.to(DEV)
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV)
    kv = dg.paged_kv4(d["k"], d["v"], d["ks"], d["vs"], td, ld, dtype=q.dtype, k_factor=kf, v_factor=vf)
    op = dg.attention4(kv, qd, out, lse=lse, q_len=q_len, window=window, sinks=sinks, scale=scale)
    ws = torch.full((dg.attn4_workspace_bytes(op),), 255, dtype=torch.uint8, device=DEV)
    dg.attn4_decode(op, ws)
    sync()
    return out, lse


def want(cache, table, lens, q, q_len=1, window=0, sinks=0, scale=None, kf=1.0, vf=1.0):
    s = float(np.float32(q.shape[2] ** -0.5 if scale is None else scale))
    n = {k: t.numpy() for k, t in cache.items()}
    f = lambda x: float(np.float32(x))
    return serve_ref.attention4(ref.f64(q), serve_ref.decode4(n["k"], n["ks"], f(kf)),
                                serve_ref.decode4(n["v"], n["vs"], f(vf)), table.numpy(), lens, q_len, s, window,
                                sinks, "f16" if q.dtype == torch.float16 else "bf16")


def check(cache, table, lens, q, what="attn4", head_major=True, **kw):
    out, lse = run(cache, table, lens, q, head_major=head_major, **kw)
    ro, rl, bo, bl = want(cache, table, lens, q, **kw)
    ref.check(ref.f64(out), ro, bo, what + " out")
    ref.check(ref.f64(lse), rl, bl, what + " lse")
    return out, lse


@pytest.mark.parametrize("ftype,heads,kv_heads,dim,page,q_len,window,sinks,head_major", [
    ("f16", 32, 8, 128, 16, 1, 0, 0, True),
    ("bf16", 12, 2, 128, 64, 1, 0, 0, True),
    ("f16", 4, 4, 64, 16, 1, 0, 0, False),
    ("bf16", 6, 1, 256, 1, 1, 0, 0, True),
    ("f16", 15, 5, 80, 24, 1, 0, 0, True),
    ("f16", 3, 1, 16, 5, 1, 0, 0, False),
    ("bf16", 20, 1, 48, 16, 1, 0, 0, True),
    ("f16", 2, 2, 192, 256, 1, 0, 0, True),
    ("f16", 33, 1, 96, 16, 1, 0, 0, True),
    ("bf16", 9, 3, 112, 16, 1, 0, 0, False),
    ("f16", 5, 1, 160, 16, 1, 0, 0, True),
    ("bf16", 16, 1, 192, 16, 3, 0, 0, False),
    ("bf16", 8, 2, 64, 16, 2, 0, 0, True),
    ("f16", 12, 2, 128, 16, 5, 0, 0, True),
    ("f16", 32, 8, 128, 64, 16, 0, 0, False),
    ("bf16", 7, 1, 256, 24, 16, 0, 0, True),
    ("f16", 4, 4, 64, 16, 1, 1, 0, True),
    ("f16", 4, 2, 64, 16, 1, 16, 4, True),
    ("bf16", 12, 2, 128, 16, 1, 100, 1, True),
    ("bf16", 4, 4, 64, 3, 8, 33, 4, True),
    ("f16", 12, 2, 128, 16, 16, 64, 70, False),
    ("f16", 5, 5, 32, 7, 3, 1, 2, True),
    ("f16", 8, 1, 128, 16, 4, 5, 0, True),
    ("bf16", 40, 8, 240, 16, 2, 50, 3, True),
])
def test_layouts_lengths_and_windows(ftype, heads, kv_heads, dim, page, q_len, window, sinks, head_major):
    need_gpu()
    cache, table = pool(LENS, page, kv_heads, dim, 3)
    q = query(len(LENS) * q_len, heads, dim, DT[ftype], 4)
    check(cache, table, LENS, q, q_len=q_len, window=window, sinks=sinks, head_major=head_major)


@pytest.mark.parametrize("ftype,q_len,window,sinks", [("f16", 1, 0, 0), ("bf16", 1, 40, 4), ("f16", 4, 0, 0),
                                                      ("bf16", 5, 40, 4)])
@pytest.mark.parametrize("dim", [64, 128, 192])
def test_nan_scales_reach_only_who_sees_them(ftype, q_len, window, sinks, dim):
    """Scales of NaN where no position lies, at later draft tokens and at positions that left
    the window; rows that see one show it in the 16 dims of its group and nowhere else."""
    need_gpu()
    lens, page = [3, 70, 129, 300], 16
    cache, table = pool(lens, page, 2, dim, 5, junk=0x7F)
    nan = 0x7F
    for b, n in enumerate(lens):
        at = lambda j: (table[b, j // page].item(), j % page)
        for j in {n - 1, max(0, n - q_len + 1)}:      # seen by some rows of the step, not by all
            cache["vs"][at(j)[0], at(j)[1], 1, dim // 16 - 1] = nan if b % 2 else 0xFF
        if b == 2:
            cache["ks"][at(n - 1)[0], at(n - 1)[1], 0, 0] = nan
        if window and n > window + q_len + sinks:     # left the window for every row, or some
            for j in (sinks, n - window - q_len, n - window - 1):
                for c in ("ks", "vs"):
                    cache[c][at(j)[0], at(j)[1]] = nan
    q = query(len(lens) * q_len, 6, dim, DT[ftype], 6)
    kw = dict(q_len=q_len, window=window, sinks=sinks)
    out, lse = run(cache, table, lens, q, **kw)
    ro, rl, bo, bl = want(cache, table, lens, q, **kw)
    assert np.isnan(ro).any() and np.isfinite(ro).any()
    ref.check(ref.f64(out), ro, bo, "out")
    ref.check(ref.f64(lse), rl, bl, "lse")


@pytest.mark.parametrize("q_len", [1, 6])
def test_missing_pages_are_unseen(q_len):
    need_gpu()
    lens, dim, page = [100, 64, 33], 128, 16
    cache, table = pool(lens, page, 2, dim, 7)
    table[0, 2] = -1
    table[0, 5] = cache["k"].shape[0]          # past the pool
    table[1, :] = -1                           # no page at all
    table[2, 1] = -7
    q = query(3 * q_len, 8, dim, torch.float16, 8)
    out, lse = check(cache, table, lens, q, q_len=q_len)
    assert (out[q_len:2 * q_len] == 0).all() and (lse[q_len:2 * q_len] == -float("inf")).all()


def test_lengths_past_the_table_and_below_zero():
    need_gpu()
    cache, table = pool([64, 64, 64], 16, 1, 64, 9)
    q = query(6, 2, 64, torch.bfloat16, 10)
    check(cache, table[:, :3], [200, 1, 49], q, q_len=2)
    out, lse = run(cache, table, [-5, -2 ** 31, 64], q, q_len=2)
    assert (out[:4] == 0).all() and (lse[:4] == -float("inf")).all() and torch.isfinite(lse[4:]).all()


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("scale,kf,vf", [(None, 0.3, 7.0), (0.0, 1.0, 1.0), (-0.2, 2.0, 0.01), (3.0, 1.0, 1e6),
                                         (1e-30, 1e-6, 1e-6), (1e-3, 1e4, 1e30)])
def test_factors_and_scales(ftype, scale, kf, vf):
    need_gpu()
    lens = [1, 40, 333]
    cache, table = pool(lens, 16, 2, 128, 11)
    q = query(3, 8, 128, DT[ftype], 12)
    if vf == 1e30 and ftype == "f16" or vf == 1e6 and ftype == "f16":
        vf = 100.0                             # fp16 ends at 65504
    check(cache, table, lens, q, scale=scale, kf=kf, vf=vf)


@pytest.mark.parametrize("size", [1e-36, 1e-8, 1e6, 1e30])
def test_queries_of_any_size_in_bf16(size):
    """Each row is taken times a power of two: the scores are those of fp32."""
    need_gpu()
    lens = [7, 200]
    cache, table = pool(lens, 16, 2, 64, 13)
    q = query(2, 6, 64, torch.float32, 14)
    q[:, ::2] *= 1e-3                          # rows of several sizes
    q = (q * size).to(torch.bfloat16)
    check(cache, table, lens, q, scale=0.1 / size)


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
def test_infinite_and_nan_queries(ftype):
    need_gpu()
    cache, table = pool([50], 16, 1, 64, 15)
    q = query(1, 4, 64, DT[ftype], 16)
    q[0, 1, 5] = float("nan")
    q[0, 2, 9] = float("inf")
    out, lse = run(cache, table, [50], q)
    assert torch.isfinite(out[0, [0, 3]]).all() and out[0, 1].isnan().all() and out[0, 2].isnan().all()
    out, lse = run(cache, table, [50], q, scale=0.0)
    assert torch.isfinite(out[0, [0, 3]]).all() and out[0, 1].isnan().all() and out[0, 2].isnan().all()


def test_weak_keys_beside_a_strong_one():
    """A thousand keys 2^-20 as strong as one: together a thousandth of the output."""
    need_gpu()
    n, dim = 1025, 64
    cache, table = pool([n], 16, 1, dim, 17)
    cache["k"].zero_()
    cache["ks"].fill_(0x38)                    # 1.0
    page, slot = table[0, 500 // 16].item(), 500 % 16
    cache["k"][page, slot, 0, 0] = 7           # one key has 7 in dim 0
    q = torch.zeros(1, 1, dim, dtype=torch.float16)
    q[0, 0, 0] = 1.0
    check(cache, table, [n], q, scale=float(20 * np.log(2) / 7))


@pytest.mark.parametrize("lens", [[20000], [3000, 1, 9000], [700] * 40, list(range(1, 300))])
def test_long_and_many_sequences_cut_between_ctas(lens):
    need_gpu()
    heads, kv, dim = 4, 2, 64
    cache, table = pool(lens, 64, kv, dim, 19)
    q = query(len(lens), heads, dim, torch.float16, 20)
    out, lse = check(cache, table, lens, q)
    again = run(cache, table, lens, q)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    for b in range(0, len(lens), max(1, len(lens) // 5)):    # a sequence alone gives the same numbers within rounding
        alone, _ = run(cache, table[b:b + 1], lens[b:b + 1], q[b:b + 1])
        assert torch.allclose(alone.float(), out[b:b + 1].float(), atol=2e-3, rtol=2e-3)


@pytest.mark.parametrize("heads,kv,dim,q_len", [(32, 8, 128, 1), (12, 2, 128, 3), (64, 8, 64, 16), (8, 2, 256, 5)])
def test_long_sequences_every_variant(heads, kv, dim, q_len):
    need_gpu()
    lens = [2500, 5, 1290]
    cache, table = pool(lens, 16, kv, dim, 21)
    q = query(len(lens) * q_len, heads, dim, torch.bfloat16, 22)
    check(cache, table, lens, q, q_len=q_len)


def test_a_cache_past_32_bit_offsets():
    """Pages whose codes and scales lie more than 2^32 bytes on."""
    need_gpu()
    pages, page, heads, dim = 70000, 64, 16, 128       # 4.6 GB of codes each for k and v
    big = {n: torch.zeros(pages, heads, page, w, dtype=torch.uint8, device=DEV) for n, w in
           (("k", dim // 2), ("v", dim // 2), ("ks", dim // 16), ("vs", dim // 16))}
    far = [69999, 33000, 2, 69998]
    n = 200
    small, _ = pool([4 * page], page, heads, dim, 23, spare=0)
    for c in big:
        for i, pg in enumerate(far):
            big[c][pg] = small[c][i].transpose(0, 1).to(DEV)
    q = query(1, 32, dim, torch.float16, 24)
    table = torch.tensor([far], dtype=torch.int32, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    out, qd = torch.empty_like(q, device=DEV), q.to(DEV)
    kv = dg.paged_kv4(*(big[c].transpose(1, 2) for c in ("k", "v", "ks", "vs")), table, lens)
    op = dg.attention4(kv, qd, out)
    dg.attn4_decode(op, torch.empty(dg.attn4_workspace_bytes(op), dtype=torch.uint8, device=DEV))
    sync()
    t = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)
    ro, _, bo, _ = want(small, t, [n], q)
    ref.check(ref.f64(out), ro, bo, "far pages")


def test_strided_q_and_out_other_streams_and_graphs():
    need_gpu()
    lens, heads, kv_heads, dim, page = [100, 37], 8, 2, 128, 16
    cache, table = pool(lens, page, kv_heads, dim, 25)
    q = query(2, heads, dim, torch.float16, 26)
    ro, _, bo, _ = want(cache, table, lens, q)
    d = {n: lay(t, True) for n, t in cache.items()}
    wide = torch.zeros(2, heads * dim * 2, dtype=torch.float16, device=DEV)
    wide[:, :heads * dim] = q.view(2, -1).to(DEV)
    qd = wide[:, :heads * dim].view(2, heads, dim)
    room = torch.full((2, heads * dim + 64), 5.0, dtype=torch.float16, device=DEV)
    out = room[:, :heads * dim].view(2, heads, dim)
    td, ld = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    kv = dg.paged_kv4(d["k"], d["v"], d["ks"], d["vs"], td, ld)
    op = dg.attention4(kv, qd, out)
    ws = torch.empty(dg.attn4_workspace_bytes(op), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dg.attn4_decode(op, ws, stream=side)
    side.synchronize()
    ref.check(ref.f64(out), ro, bo, "side stream")
    assert (room[:, heads * dim:] == 5).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.attn4_decode(op, ws)
    for n in ([60, 37], [100, 1], [0, 20]):             # the graph follows the lengths
        ld.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        sync()
        ro, _, bo, _ = want(cache, table, n, q)
        ref.check(ref.f64(out), ro, bo, "graph")


@pytest.mark.parametrize("dim,off", [(128, 4), (128, 8), (96, 1), (64, 2), (256, 4)])
def test_scales_anywhere_and_codes_at_eight_bytes(dim, off):
    """Scale rows at odd addresses, code rows at multiples of eight."""
    need_gpu()
    lens, heads, kv_heads, page = [70, 33], 4, 2, 16
    cache, table = pool(lens, page, kv_heads, dim, 27)
    q = query(2, heads, dim, torch.float16, 28)
    d = {}
    for n, t in cache.items():
        w, room = t.shape[3], off if n in ("ks", "vs") else 8
        flat = torch.full((t.shape[0] * page * kv_heads * (w + room) + 64,), 0x7F, dtype=torch.uint8, device=DEV)
        v = flat[room:room + t.shape[0] * page * kv_heads * (w + room)].view(t.shape[0], page, kv_heads, w + room)[..., :w]
        v.copy_(t)
        d[n] = v
    td, ld, qd = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), q.to(DEV)
    out = torch.empty_like(qd)
    kv = dg.paged_kv4(d["k"], d["v"], d["ks"], d["vs"], td, ld)
    op = dg.attention4(kv, qd, out)
    dg.attn4_decode(op, torch.empty(dg.attn4_workspace_bytes(op), dtype=torch.uint8, device=DEV))
    sync()
    ro, _, bo, _ = want(cache, table, lens, q)
    ref.check(ref.f64(out), ro, bo, "odd places")


@pytest.mark.parametrize("vf,lo,hi", [(1e36, 0x01, 0x18), (1e37, 0x01, 0x08), (3e-37, 0x60, 0x7F), (1e-36, 0x38, 0x40),
                                      (1e30, 0x20, 0x38)])
@pytest.mark.parametrize("lens", [[20000], [100, 5000, 3], [40]])
def test_value_factors_at_the_ends(vf, lo, hi, lens):
    """Values that bf16 holds: neither the weights' sum in front of the factor nor the factor over that sum may leave
    fp32's range, in sequences of one part and of many."""
    need_gpu()
    cache, table = pool(lens, 16, 1, 128, 21, lo=lo, hi=hi)
    cache["ks"] = torch.full_like(cache["ks"], 0x28)
    q = query(len(lens), 4, 128, torch.bfloat16, 22)
    check(cache, table, lens, q, vf=vf)
