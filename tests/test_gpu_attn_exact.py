"""Attention to the precision that the header states: fp32 scores and sums, weights
2^-21 (fp16) or 2^-16 (bf16) off, one rounding into the output; infinities and NaN
that a token does see follow IEEE."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
WEIGHT = {"f16": 2.0 ** -21, "bf16": 2.0 ** -16}   # of a weight, as the sum of two 16-bit numbers
LEAST = {"f16": 2.0 ** -32, "bf16": 0.0}           # what may be lost of one, next to the strongest


def _attention(q, k, v, lens, ftype, q_len=1, page=16, window=0, sinks=0, scale=None):
    """q [T][H][D]; k, v [n][G][D]: every sequence reads the same n positions.
    Returns out and lse."""
    n, G, D = k.shape
    pages = -(-n // page)
    pool = torch.zeros(2, pages * page, G, D, dtype=q.dtype)
    pool[0, :n], pool[1, :n] = k, v
    pool = pool.view(2, pages, page, G, D).to(DEV)
    table = torch.arange(pages, dtype=torch.int32).repeat(len(lens), 1).to(DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qd = q.to(DEV)
    out = torch.full_like(qd, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV)
    op = dg.attention(dg.paged_kv(pool[0], pool[1], table, ld), qd, out, lse=lse, q_len=q_len, window=window,
                      sinks=sinks, scale=scale)
    ws = torch.full((dg.attn_workspace_bytes(op),), 255, dtype=torch.uint8, device=DEV)
    dg.attn_decode(op, ws)
    sync()
    return ref.f64(out), ref.f64(lse)


def _exact(q, k, v, keep, ftype, scale=None):
    """One row q [D] over the positions `keep` of k, v [n][D], in 64 bits: out, lse
    and their bounds."""
    q, k, v = ref.f64(q), ref.f64(k)[keep], ref.f64(v)[keep]
    D, n, scale = q.size, len(keep), q.size ** -0.5 if scale is None else float(np.float32(scale))
    z = scale * (k @ q)
    m = z.max()
    e = np.exp(z - m)
    l = e.sum()
    with np.errstate(invalid="ignore"):
        out = e @ v / l
        A = e @ np.abs(v) / l
        lost = LEAST[ftype] * np.abs(v).sum(0) / l
    lse = m + np.log(l)
    ez = ((D + 2) * ref.U32 * abs(scale) * (np.abs(k) @ np.abs(q)) + ref.U32 * np.abs(z)).max()
    rel = ez + ref.FN + (n + 2) * ref.U32
    bound = A * (2 * rel + WEIGHT[ftype]) + lost + ref.U16[ftype] * np.abs(out) + ref.TINY[ftype]
    return out, lse, bound, rel + ref.FN + 2 * ref.U32 * (abs(m) + abs(lse))


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,n,q_len", [(4, 2, 64, 40, 1), (32, 2, 64, 600, 4), (8, 2, 128, 333, 1),
                                                        (40, 2, 128, 90, 2), (3, 1, 192, 257, 1), (5, 1, 256, 64, 2)])
def test_weights_keep_more_than_one_rounding(ftype, heads, kv_heads, dim, n, q_len):
    """Values in pairs of opposite sign under nearly equal weights: the output is a
    small difference of large sums, where rounded weights would show."""
    need_gpu()
    g = torch.Generator().manual_seed(dim + n)
    k = torch.randn(n, kv_heads, dim, generator=g).to(DT[ftype])
    v = torch.randn(n, kv_heads, dim, generator=g).to(DT[ftype])
    v[1::2] = -v[0:n - 1:2]
    q = (torch.randn(q_len, heads, dim, generator=g) * 0.03).to(DT[ftype])
    out, lse = _attention(q, k, v, [n], ftype, q_len)
    for t in range(q_len):
        for h in range(heads):
            kv = h // (heads // kv_heads)
            ro, rl, bo, bl = _exact(q[t, h], k[:, kv], v[:, kv], np.arange(n - q_len + t + 1), ftype)
            ref.check(out[t, h], ro, bo, "out of token %d, head %d" % (t, h))
            ref.check(lse[t, h], rl, bl, "lse of token %d, head %d" % (t, h))


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
def test_many_weak_keys_beside_a_strong_one(ftype):
    """2048 keys of weight e^-17 beside one strong key whose value is zero: their sum
    is the output.  64 sequences of 8 heads, so that one warp reads hundreds of them."""
    need_gpu()
    n, G, D, B = 2049, 8, 64, 64
    k, v = torch.zeros(n, G, D, dtype=DT[ftype]), torch.full((n, G, D), 30000.0).to(DT[ftype])
    k[5, :, 0], v[5] = 17.0 * 8, 0.0                     # 17 / scale / q
    q = torch.zeros(B, G, D, dtype=DT[ftype])
    q[:, :, 0] = 1.0
    out, lse = _attention(q, k, v, [n] * B, ftype)
    ro, rl, bo, bl = _exact(q[0, 0], k[:, 0], v[:, 0], np.arange(n), ftype)
    ref.check(out, np.broadcast_to(ro, out.shape), bo, "out")
    ref.check(lse, np.broadcast_to(rl, lse.shape), bl, "lse")


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("q_len,window", [(1, 0), (3, 0), (2, 50)])
def test_infinities_and_nan_that_a_token_sees(ftype, q_len, window):
    """One visible value of each kind, in dims of its own: the output is that
    infinity or NaN in the dim and unharmed beside it."""
    need_gpu()
    n, D, inf = 150, 64, float("inf")
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn(n, 1, D, generator=g).to(DT[ftype]) for _ in range(2))
    q = (torch.randn(q_len, 4, D, generator=g) * 2).to(DT[ftype])
    for j, d, x in ((120, 0, inf), (121, 1, -inf), (122, 2, float("nan")), (123, 3, inf), (n - 1, 3, inf),
                    (130, 4, -inf), (131, 4, inf), (n - q_len, 5, -inf), (n - 1, 6, inf), (3, 7, inf)):
        v[j, 0, d] = x
    out, lse = _attention(q, k, v, [n], ftype, q_len, window=window)
    for t in range(q_len):
        p = n - q_len + t
        keep = np.arange(max(0, p - window + 1) if window else 0, p + 1)
        for h in range(4):
            with np.errstate(invalid="ignore"):
                ro, rl, bo, bl = _exact(q[t, h], k[:, 0], v[:, 0], keep, ftype)
            assert np.isinf(ro).any() and np.isnan(ro).any() and np.isfinite(ro).any()
            ref.check(out[t, h], ro, bo, "out of token %d, head %d" % (t, h))
            ref.check(lse[t, h], rl, bl, "lse of token %d, head %d" % (t, h))


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-45, 3e-39, -1e-38, 1.5e-38, 1e-30])
def test_tiny_scales_weigh_all_positions_alike(ftype, scale):
    need_gpu()
    n, D = 300, 64
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(n, 1, D, generator=g).to(DT[ftype]) for _ in range(2))
    q = torch.randn(1, 2, D, generator=g).to(DT[ftype])
    out, lse = _attention(q, k, v, [n], ftype, scale=scale)
    for h in range(2):
        ro, rl, bo, bl = _exact(q[0, h], k[:, 0], v[:, 0], np.arange(n), ftype, scale)
        ref.check(out[0, h], ro, bo, "out of head %d" % h)
        ref.check(lse[0, h], rl, bl, "lse of head %d" % h)


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("n,scale,large", [(300, -1e30, 1.0), (300, 1e10, 1.0), (9000, 1e20, 1.0), (300, None, 3000.0),
                                           (9000, None, 60000.0)])
def test_large_scores_leave_the_strongest_position(ftype, n, scale, large):
    """Scores far past 2^24, where fp32 holds them to whole numbers and worse, but the
    strongest lies further from the rest than that."""
    need_gpu()
    D = 64
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(n, 1, D, generator=g).to(DT[ftype]) for _ in range(2))
    q = (torch.randn(1, 2, D, generator=g) * large).clamp(-60000, 60000).to(DT[ftype])
    k = (k * large).clamp(-60000, 60000).to(DT[ftype])
    out, lse = _attention(q, k, v, [n], ftype, scale=scale)
    scale = D ** -0.5 if scale is None else float(np.float32(scale))
    for h in range(2):
        z = scale * (ref.f64(k[:, 0]) @ ref.f64(q[0, h]))
        err = (D + 3) * ref.U32 * abs(scale) * (np.abs(ref.f64(k[:, 0])) @ np.abs(ref.f64(q[0, h]))).max()
        assert np.sort(z)[-2] < z.max() - 2 * err - 200      # the others weigh nothing
        assert np.array_equal(out[0, h], ref.f64(v[z.argmax(), 0]))
        assert abs(lse[0, h] - z.max()) <= err + 4 * ref.U32 * abs(z.max())


def test_lengths_and_tables_that_the_kernel_before_writes():
    """The length is a greedy token and the page table an expert layer's choice, each
    written by the library's own kernel right before the append and the attention, which
    start while it still runs: 64 different ones in a row, then compared."""
    need_gpu()
    g = torch.Generator().manual_seed(11)
    steps, pages, page, G, D, K = 64, 12, 16, 2, 64, 64
    f16 = lambda *s: torch.randn(*s, generator=g).half()
    vocab = page * 8
    lengths = 1 + torch.randperm(vocab - 1, generator=g)[:steps]                     # 1 .. 127
    order = torch.stack([torch.randperm(pages, generator=g)[:8] for _ in range(steps)])
    code = torch.linalg.qr(torch.randn(vocab, vocab, generator=g, dtype=torch.float64))[0]
    head = code.half()                                                               # row j answers to column j
    xs = head[lengths]
    mark = torch.zeros(steps, K)                                                     # x picks its experts in order
    mark.scatter_(1, order, torch.linspace(9, 2, 8).repeat(steps, 1))
    router = torch.eye(pages, K).half()
    k, v, q = f16(pages, page, G, D), f16(pages, page, G, D), f16(steps, 4, D)
    kn, vn = f16(steps, G, D), f16(steps, G, D)

    on = lambda t: t.contiguous().to(DEV)
    kd, vd, qd, xd, md, hd, rd, knd, vnd = (on(t) for t in (k, v, q, xs, mark.half(), head, router, kn, vn))
    length, table = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (1, 8))
    out = torch.empty(steps, 4, D, dtype=torch.float16, device=DEV)
    logits = torch.empty(vocab, dtype=torch.float32, device=DEV)
    w = [on(f16(pages, 32, K)), on(f16(pages, 32, K)), on(f16(pages, K, 32))]
    y = torch.empty(K, dtype=torch.float16, device=DEV)
    kv = dg.paged_kv(kd, vd, table.view(1, 8), length)
    ops = []
    for i in range(steps):
        ops.append((dg.moe(dg.LINEAR_F16, md[i], y, rd, *w, 8, ids=table),
                    dg.linear(dg.LINEAR_F16, hd, 1, vocab, vocab, x=xd[i], logits=logits, token=length),
                    dg.append(kv, None, knd[i:i + 1], vnd[i:i + 1]), dg.attention(kv, qd[i:i + 1], out[i:i + 1])))
    new = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    ws_m, ws_h = new(dg.moe_workspace_bytes(ops[0][0])), new(dg.workspace_bytes([ops[0][1]]))
    ws_a = new(dg.attn_workspace_bytes(ops[0][3]))
    for experts, greedy, append, attend in ops:
        dg.moe_forward(experts, ws_m)
        dg.lm_head_argmax(greedy, ws_h)
        dg.kv_append(append)
        dg.attn_decode(attend, ws_a)
    sync()
    kh, vh = ref.f64(k), ref.f64(v)
    for i in range(steps):
        n, ids = int(lengths[i]), order[i].numpy()
        _, kh, vh, _, _ = ref.append(np.zeros((1, 0, D)), ref.f64(kn[i:i + 1]), ref.f64(vn[i:i + 1]), kh, vh, ids[None],
                                     [n], 1, None, None, False, "f16")
        flat = kh[ids].reshape(-1, G, D), vh[ids].reshape(-1, G, D)
        for h in range(4):
            ro, _, bo, _ = _exact(q[i, h], torch.from_numpy(flat[0][:, h // 2]), torch.from_numpy(flat[1][:, h // 2]),
                                  np.arange(n), "f16")
            ref.check(ref.f64(out[i, h]), ro, bo, "step %d, head %d" % (i, h))
    assert np.array_equal(ref.f64(kd), kh) and np.array_equal(ref.f64(vd), vh)


@pytest.mark.parametrize("rot", [0, 32])
def test_append_at_the_most_negative_length(rot):
    """No token has a position: zeros in q_out, nothing in the cache."""
    need_gpu()
    g = torch.Generator().manual_seed(12)
    f16 = lambda *s: torch.randn(*s, generator=g).half().to(DEV)
    k_cache, v_cache, q, k, v = f16(4, 16, 2, 64), f16(4, 16, 2, 64), f16(6, 4, 64), f16(6, 2, 64), f16(6, 2, 64)
    kh, vh = k_cache.clone(), v_cache.clone()
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    lens = torch.tensor([-2 ** 31, -2 ** 31 + 1], dtype=torch.int32, device=DEV)
    cos = sin = None
    if rot:
        cos = sin = torch.ones(32, rot // 2, device=DEV)
    q_out = torch.full_like(q, 7.0)
    dg.kv_append(dg.append(dg.paged_kv(k_cache, v_cache, table, lens), q, k, v, q_out, q_len=3, cos=cos, sin=sin))
    sync()
    assert (q_out == 0).all() and torch.equal(k_cache, kh) and torch.equal(v_cache, vh)


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 0.125])
def test_infinite_and_nan_queries_are_nan_at_any_scale(ftype, scale):
    need_gpu()
    n, D = 90, 64
    g = torch.Generator().manual_seed(13)
    k, v = (torch.randn(n, 1, D, generator=g).to(DT[ftype]) for _ in range(2))
    q = torch.randn(1, 5, D, generator=g).to(DT[ftype])
    q[0, 1, 7], q[0, 2, 7], q[0, 3, 7] = float("nan"), float("inf"), -float("inf")
    out, lse = _attention(q, k, v, [n], ftype, scale=scale)
    for h in (0, 4):
        ro, rl, bo, bl = _exact(q[0, h], k[:, 0], v[:, 0], np.arange(n), ftype, scale)
        ref.check(out[0, h], ro, bo, "out of head %d" % h)
        ref.check(lse[0, h], rl, bl, "lse of head %d" % h)
    assert np.isnan(out[0, 1]).all() and np.isnan(lse[0, 1])
    for h in (2, 3):      # scores of +-infinity (their softmax: inf - inf), or 0 * inf
        assert np.isnan(out[0, h]).all()


@pytest.mark.parametrize("ftype,small", [("f16", 2.0 ** -24), ("bf16", 2.0 ** -133)])
def test_subnormal_queries_count(ftype, small):
    """The smallest numbers of the type, under a scale that makes them matter."""
    need_gpu()
    n, D, scale = 40, 64, -2.0 ** 14 if ftype == "f16" else -2.0 ** 100
    g = torch.Generator().manual_seed(14)
    k, v = (torch.randn(n, 1, D, generator=g) for _ in range(2))
    k = (k * (1.0 if ftype == "f16" else 2.0 ** 30)).to(DT[ftype])
    v = v.to(DT[ftype])
    q = (torch.randint(-40, 41, (1, 3, D), generator=g) * small).to(DT[ftype])
    out, lse = _attention(q, k, v, [n], ftype, scale=scale)
    for h in range(3):
        ro, rl, bo, bl = _exact(q[0, h], k[:, 0], v[:, 0], np.arange(n), ftype, scale)
        assert np.abs(rl - np.log(n)) > 1e-3
        ref.check(out[0, h], ro, bo, "out of head %d" % h)
        ref.check(lse[0, h], rl, bl, "lse of head %d" % h)
