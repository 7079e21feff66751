"""Head norms, rotation and the append (dg_qkv_append) to 16-bit and 4-bit caches, by lengths and
by slots, and the 4-bit cache read back (dg_kv4_read), against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
import serve_ref
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = float(np.float32(1e-5))


class Case:
    """A cache (its bytes marked), q, k and v as columns of one product's rows, and a run on them."""

    def __init__(self, ftype, bits, heads, kvh, dim, page, lens, q_len=0, seed=0, rot=None, inter=False, layer=False,
                 norm="qk", w_offset=0.0, kf=1.0, vf=1.0, max_pos=None, by_map=False, odd=0, std=1.0):
        self.__dict__.update({k: v for k, v in locals().items() if k != "self"})
        g = torch.Generator().manual_seed(seed)
        dt, B = DT[ftype], len(lens)
        used = [max(1, -(-max(n, 0) // page)) for n in lens]
        P = sum(used) + 2
        order = torch.randperm(P, generator=g).int()
        self.table = torch.full((B, max(used) + 1), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
        if by_map:
            self.pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int64)
            seq = np.repeat(np.arange(B), lens)
        else:
            self.pos = np.array([n - q_len + i for n in np.maximum(lens, 0) for i in range(q_len)])
            seq = np.repeat(np.arange(B), q_len)
        T = len(self.pos)
        pages = [int(self.table[s, p // page]) if p >= 0 and p // page < self.table.shape[1] else -1
                 for s, p in zip(seq, self.pos)]
        self.slot = np.array([pg * page + p % page if pg >= 0 else -1 for pg, p in zip(pages, self.pos)], np.int64)
        width = (heads + 2 * kvh) * dim + 2 * odd
        qkv = (torch.randn(T, width, generator=g) * std).to(dt)
        cut = lambda a, n: qkv[:, odd + a * dim:odd + (a + n) * dim].reshape(T, n, dim)
        self.q, self.k, self.v = cut(0, heads), cut(heads, kvh), cut(heads + kvh, kvh)
        self.qkv = qkv
        rot = dim if rot is None else rot
        top = max(max(lens), 1) + 3 if max_pos is None else max_pos
        ang = torch.arange(top, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(rot // 2).double() / max(rot, 1))
        self.cos, self.sin = (ang.cos().float(), ang.sin().float()) if rot else (None, None)
        self.w_q = (1 + 0.3 * torch.randn(dim, generator=g)).to(dt) if "q" in norm and heads else None
        self.w_k = (1 + 0.3 * torch.randn(dim, generator=g)).to(dt) if "k" in norm else None
        if bits == 16:
            self.cache = [torch.full((P, page, kvh, dim), 9.0, dtype=dt) for _ in "kv"]
        else:
            self.cache = [torch.full((P, page, kvh, w), 0x5A, dtype=torch.uint8) for w in (dim // 2, dim // 2, dim // 16,
                                                                                          dim // 16)]

    def run(self, head_major=True, in_place=False, stream=None):
        dev = lambda t: None if t is None else t.to(DEV)
        place = (lambda t: t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)) if head_major else dev
        qkv = self.qkv.to(DEV)
        o, T = self.odd, len(self.pos)
        cut = lambda a, n: qkv[:, o + a * self.dim:o + (a + n) * self.dim].view(T, n, self.dim)
        q, k, v = cut(0, self.heads), cut(self.heads, self.kvh), cut(self.heads + self.kvh, self.kvh)
        room = torch.full((T, self.heads * self.dim + 2 * o + 8), 5.0, dtype=self.qkv.dtype, device=DEV)
        q_out = q if in_place else room[:, o:o + self.heads * self.dim].view(T, self.heads, self.dim)
        cache, table = [place(t) for t in self.cache], dev(self.table)
        lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        if self.bits == 16:
            kv = dg.paged_kv(*cache, table, lens)
        else:
            kv = dg.paged_kv4(*cache, table, lens, dtype=self.qkv.dtype, k_factor=self.kf, v_factor=self.vf)
        slots = torch.from_numpy(self.slot).to(DEV) if self.by_map else None
        where = (dict(slots=slots, positions=torch.from_numpy(self.pos).int().to(DEV)) if self.by_map else
                 dict(q_len=self.q_len))
        keep = [dev(t) for t in (self.cos, self.sin, self.w_q, self.w_k)]
        op = dg.head_append(kv, q if self.heads else None, k, v, q_out if self.heads else None, cos=keep[0], sin=keep[1],
                            interleaved=self.inter, w_q=keep[2], w_k=keep[3], eps=EPS, w_offset=self.w_offset,
                            kind=dg.NORM_LAYER if self.layer else dg.NORM_RMS, **where)
        dg.qkv_append(op, stream=stream)
        sync()
        got = {"q": q_out.clone(), "cache": [t.cpu() for t in cache]}
        if not in_place:
            assert (room[:, o + self.heads * self.dim:] == 5).all() and (room[:, :o] == 5).all()
            assert torch.equal(qkv.cpu().view(torch.int16), self.qkv.view(torch.int16))
        if self.bits == 4:
            kr, vr = (torch.full((T, self.kvh, self.dim), 7.0, dtype=self.qkv.dtype, device=DEV) for _ in "kv")
            dg.kv4_read(dg.kv4_rows(kv, kr, vr, **({"slots": slots} if self.by_map else where)))
            sync()
            got["read"] = kr.cpu(), vr.cpu()
        return got

    def check(self, **kw):
        got = self.run(**kw)
        f = lambda t: None if t is None else ref.f64(t)
        q, eq, k, ek, live = serve_ref.head_append(f(self.q), f(self.k), f(self.w_q), f(self.w_k), EPS,
                                                   float(np.float32(self.w_offset)), self.layer, self.pos, f(self.cos),
                                                   f(self.sin), self.inter)
        u, tiny = ref.U16[self.ftype], ref.TINY[self.ftype]
        if self.heads:
            ref.check(ref.f64(got["q"]), q, eq + u * (np.abs(q) + eq) + tiny, "q")
        v, written = f(self.v), live & (self.slot >= 0)
        P, page = self.cache[0].shape[:2]
        hit = np.zeros(P * page, bool)
        hit[self.slot[written]] = True
        for c, was in zip(got["cache"], self.cache):     # what no token owns is as it was
            same = (c == was).reshape(P * page, -1).all(1).numpy()
            assert same[~hit].all(), "a place that no token owns"
        at = self.slot[written]
        if self.bits == 16:
            kc, vc = (ref.f64(c).reshape(P * page, self.kvh, self.dim)[at] for c in got["cache"])
            ref.check(kc, k[written], (ek + u * (np.abs(k) + ek) + tiny)[written], "keys")
            assert np.array_equal(vc, v[written], equal_nan=True)
            return got
        n = [c.numpy().reshape(P * page, self.kvh, c.shape[3])[at] for c in got["cache"]]
        for name, codes, scales, x, ex, fac, read in (("k", n[0], n[2], k, ek, self.kf, got["read"][0]),
                                                      ("v", n[1], n[3], v, np.zeros_like(v), self.vf, got["read"][1])):
            fac = float(np.float32(fac))
            held = serve_ref.decode4(codes, scales, fac)
            want = [serve_ref.coded(x[t], ex[t], fac) for t in np.flatnonzero(written)]
            if len(want):
                ref.check(held, np.stack([w[0] for w in want]), np.stack([w[1] for w in want]), name + " held")
            nib = np.stack((codes & 15, codes >> 4))
            assert (nib != 8).all(), "a code of -8"
            back = np.zeros_like(x)
            there = self.slot >= 0
            flat = [c.numpy().reshape(P * page, self.kvh, c.shape[3])[self.slot[there]] for c in got["cache"]]
            i = 0 if name == "k" else 1
            back[there] = serve_ref.decode4(flat[i], flat[2 + i], fac)
            ref.check(ref.f64(read), back, u * np.abs(back) * 1.001 + tiny, name + " read")
        return got


LENS = [0, 1, 2, 5, 16, 17, 40]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("ftype,heads,kvh,dim,page,q_len,rot,inter,layer", [
    ("f16", 12, 2, 128, 16, 1, None, False, False),
    ("bf16", 32, 8, 128, 16, 4, 64, True, False),
    ("f16", 4, 4, 64, 64, 2, None, False, True),
    ("bf16", 5, 1, 256, 5, 16, 128, False, True),
    ("f16", 15, 5, 80, 24, 1, 32, False, False),
    ("bf16", 3, 3, 96, 1, 3, 0, False, True),
    ("f16", 2, 2, 192, 16, 2, None, True, False),
    ("bf16", 1, 1, 16, 16, 1, 16, False, False),
    ("f16", 7, 1, 48, 16, 2, 20, False, False),        # pairs that no 16 bytes hold
    ("bf16", 6, 2, 112, 16, 5, 2, True, False),
    ("f16", 0, 3, 128, 16, 1, None, False, False),     # no q
    ("f16", 28, 4, 240, 16, 1, 240, False, True),
])
def test_layouts(bits, ftype, heads, kvh, dim, page, q_len, rot, inter, layer):
    need_gpu()
    Case(ftype, bits, heads, kvh, dim, page, LENS, q_len, 1, rot, inter, layer, kf=0.5, vf=2.0).check(
        head_major=dim % 128 == 0)


@pytest.mark.parametrize("dim", [8, 24, 40, 136])
def test_16_bit_heads_of_other_multiples_of_eight(dim):
    need_gpu()
    Case("f16", 16, 5, 2, dim, 16, LENS, 3, 2).check()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("norm", ["", "q", "k"])
def test_only_some_are_normed(bits, norm):
    need_gpu()
    Case("bf16", bits, 6, 2, 64, 16, LENS, 2, 3, norm=norm, w_offset=1.0).check()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("odd", [1, 3, 8])
def test_rows_that_start_anywhere(bits, odd):
    need_gpu()
    Case("f16", bits, 6, 2, 128, 16, LENS, 2, 4, odd=odd).check(head_major=False)


@pytest.mark.parametrize("bits", [16, 4])
def test_in_place(bits):
    need_gpu()
    a = Case("bf16", bits, 12, 2, 128, 16, LENS, 2, 5)
    assert torch.equal(a.run(in_place=True)["q"], a.check()["q"])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens", [[1], [33, 1, 200, 7], [0, 5, 0, 12]])
def test_prompts_by_slots(bits, lens):
    need_gpu()
    c = Case("f16", bits, 12, 2, 128, 16, lens, by_map=True, seed=6)
    c.check()
    past = c.cache[0].shape[0] * 16
    c.slot[::3] = -1                         # tokens that were given no place
    c.slot[1::7] = past + np.maximum(c.slot[1::7], 0)      # and ones past the pool
    c.pos[2::5] = -1
    got = c.run()
    assert (got["q"][torch.from_numpy(c.pos < 0).to(DEV)] == 0).all()
    c.slot[c.slot >= past] = -1              # the same for the cache
    same = c.check()
    assert torch.equal(got["q"], same["q"]) and all(torch.equal(a, b) for a, b in zip(got["cache"], same["cache"]))


@pytest.mark.parametrize("bits", [16, 4])
def test_past_the_tables(bits):
    """Positions past cos and sin, or past the block table, or in a page that is missing."""
    need_gpu()
    c = Case("f16", bits, 4, 2, 64, 16, [30, 12, 18, 40], 8, 7, max_pos=36)
    c.check()
    c = Case("f16", bits, 4, 2, 64, 16, [30, 12, 18, 40], 8, 7)
    c.table[3, 2] = -1
    c.table[0, 1] = c.cache[0].shape[0]
    gone = np.zeros(len(c.pos), bool)
    for b, i in ((3, 2), (0, 1)):
        for t in range(b * 8, b * 8 + 8):
            gone[t] |= c.pos[t] // 16 == i
    c.slot[gone] = -1
    c.check()
    c = Case("f16", bits, 4, 2, 64, 16, [-3, -2 ** 31, 5], 2, 8)
    c.check()


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
def test_4_bit_groups_at_the_ends(ftype):
    """Groups of zeros, of values too small or too large for a scale, of infinities and NaN, and
    halves of a step (which go to the even code)."""
    need_gpu()
    c = Case(ftype, 4, 0, 2, 128, 16, [9], 9, 9, rot=0, norm="")
    for x in (c.k, c.v):
        x[0] = 0
        x[1] = x[1] * 1e-3                        # scales below 2^-6 lose bits
        x[2] = x[2] * 1e-4                        # scales of one or two steps
        x[3, :, :16] = 2.0 ** -20                 # no scale at all
        x[4] = x[4] * 3000                        # past 448 x 7: clipped
        x[5, 0, 3] = float("nan")
        x[6, 1, 100] = float("inf")
        x[7, 0, 127] = -float("inf")
        x[8] = torch.arange(256).view(2, 128).remainder(29).sub(14).to(x.dtype) * 0.5    # amax 7: step 1, halves
    c.qkv = torch.cat((c.k.reshape(9, -1), c.v.reshape(9, -1)), 1)
    got = c.check()
    at = c.slot[8]
    codes = got["cache"][1].reshape(-1, 2, 64)[at].numpy()
    scales = got["cache"][3].reshape(-1, 2, 8)[at].numpy()
    x = ref.f64(c.v[8]).reshape(2, 8, 16)
    exact = np.abs(x).max(-1) == 7.0
    assert (scales[exact] == 0x38).all() and exact.sum() >= 8
    held = serve_ref.decode4(codes, scales, 1.0).reshape(2, 8, 16)
    assert np.array_equal(held[exact], np.clip(np.round(x[exact]), -7, 7))
    s = got["cache"][3].reshape(-1, 2, 8)[c.slot[5:8]].numpy()
    assert s[0, 0, 0] == 0x7F and s[1, 1, 6] == 0x7F and s[2, 0, 7] == 0x7F and (s == 0x7F).sum() == 3


@pytest.mark.parametrize("bits", [16, 4])
def test_values_that_cancel(bits):
    """A mean far above the spread: the centred norm takes it off before it squares."""
    need_gpu()
    c = Case("f16", bits, 4, 2, 128, 16, [20], 4, 10, layer=True)
    c.qkv.add_(100.0)
    cut = lambda a, n: c.qkv[:, a * 128:(a + n) * 128].reshape(-1, n, 128)
    c.q, c.k, c.v = cut(0, 4), cut(4, 2), cut(6, 2)
    c.check()


def test_graphs_follow_lengths_and_other_streams():
    need_gpu()
    c = Case("f16", 4, 4, 2, 64, 16, [20, 33], 1, 11)
    dev = lambda t: t.to(DEV)
    cache, table, lens = [dev(t) for t in c.cache], dev(c.table), torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    kv = dg.paged_kv4(*cache, table, lens)
    q, k, v, q_out = dev(c.q), dev(c.k), dev(c.v), torch.empty(2, 4, 64, dtype=torch.float16, device=DEV)
    cos, sin, w_q, w_k = (dev(t) for t in (c.cos, c.sin, c.w_q, c.w_k))
    op = dg.head_append(kv, q, k, v, q_out, cos=cos, sin=sin, w_q=w_q, w_k=w_k, eps=EPS)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.qkv_append(op)
    for n in ([20, 33], [7, 1], [0, 18]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for t in cache:
            t.fill_(0x5A)
        graph.replay()
        sync()
        by_graph, q_graph = [t.clone() for t in cache], q_out.clone()
        for t in cache:
            t.fill_(0x5A)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        dg.qkv_append(op, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(by_graph, cache)) and torch.equal(q_graph, q_out)
        page, at = c.table[1, (n[1] - 1) // 16].item(), (n[1] - 1) % 16
        assert (cache[0][page, at] != 0x5A).any()


def test_read_of_whole_sequences_and_one_side():
    """q_len of any size: a sequence's cache from its start on, zeros before it."""
    need_gpu()
    r = np.random.RandomState(12)
    codes = torch.from_numpy(r.randint(0, 256, (7, 16, 2, 32)).astype(np.uint8))
    scales = torch.from_numpy(r.randint(0, 256, (7, 16, 2, 4)).astype(np.uint8))      # negative and NaN ones too
    table = torch.tensor([[3, 0, 5], [6, -1, 2]], dtype=torch.int32)
    lens = [41, 44]
    keep, L = [t.to(DEV) for t in (codes, scales, table)], 50
    lens_d = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kv = dg.paged_kv4(keep[0], keep[0], keep[1], keep[1], keep[2], lens_d, k_factor=0.7)
    k = torch.full((2 * L, 2, 64), 3.0, dtype=torch.float16, device=DEV)
    dg.kv4_read(dg.kv4_rows(kv, k, None, q_len=L))
    sync()
    want = np.zeros((2, L, 2, 64))
    values = serve_ref.decode4(codes.numpy(), scales.numpy(), float(np.float32(0.7)))
    for b, n in enumerate(lens):
        for p in range(n):
            page = int(table[b, p // 16])
            if page >= 0:
                want[b, L - n + p] = values[page, p % 16]
    ref.check(ref.f64(k).reshape(want.shape), want, ref.U16["f16"] * np.abs(want) * 1.001 + ref.TINY["f16"], "read")


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("ftype,heads,kvh,dim,rot,inter,layer,tokens", [
    ("f16", 12, 3, 128, None, False, True, 700),
    ("bf16", 9, 1, 256, 64, False, False, 560),        # lanes with and without a pair in a team
    ("f16", 20, 5, 64, 32, False, False, 800),
    ("bf16", 20, 5, 64, 16, False, True, 800),         # half of a scale group
    ("f16", 17, 2, 96, 96, False, False, 560),
    ("bf16", 13, 4, 80, 48, False, True, 560),
    ("f16", 10, 5, 192, None, True, False, 300),
    ("bf16", 12, 4, 128, 0, False, True, 560),
    ("f16", 0, 18, 112, 96, False, False, 300),
    ("bf16", 3, 1, 16, 16, False, False, 4200),
    ("f16", 3, 1, 32, 32, False, True, 4200),
])
def test_many_tokens(bits, ftype, heads, kvh, dim, rot, inter, layer, tokens):
    """More heads than the GPU has warps for at a time, in prompts that end inside pages."""
    need_gpu()
    c = Case(ftype, bits, heads, kvh, dim, 16, [1, tokens // 2, 3, tokens - tokens // 2 - 4], seed=11, rot=rot, inter=inter,
             layer=layer, by_map=True, kf=0.5, vf=2.0)
    got = c.check()
    if heads:
        assert torch.equal(c.run(in_place=True)["q"], got["q"])


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("factor", [1e37, 4e36, 1e33, 1.0, 1e-30, 1e-37])
def test_read_with_factors_at_the_ends(ftype, factor):
    """Codes of zero are zeros under every scale that is a number, also where scale and factor pass fp32."""
    need_gpu()
    r = np.random.RandomState(13)
    codes = torch.from_numpy(r.choice([0, 0x10, 0x0F, 0x80, 0x71, 0x90], (5, 16, 2, 32)).astype(np.uint8))
    scales = torch.from_numpy(r.choice([0, 1, 0x38, 0x7D, 0x7E, 0xFE, 0x7F], (5, 16, 2, 4)).astype(np.uint8))
    table, lens = torch.arange(5, dtype=torch.int32, device=DEV).view(1, 5), torch.tensor([80], dtype=torch.int32, device=DEV)
    c, s = codes.to(DEV), scales.to(DEV)
    kv = dg.paged_kv4(c, c, s, s, table, lens, dtype=DT[ftype], k_factor=factor, v_factor=factor)
    out = [torch.full((80, 2, 64), 3.0, dtype=DT[ftype], device=DEV) for _ in "kv"]
    dg.kv4_read(dg.kv4_rows(kv, *out, q_len=80))
    sync()
    want = serve_ref.decode4(codes.numpy(), scales.numpy(), float(np.float32(factor))).reshape(80, 2, 64)
    most = torch.finfo(DT[ftype]).max * (1 + ref.U16[ftype])       # rounds to infinity from here on
    with np.errstate(invalid="ignore"):
        want = np.where(np.abs(want) >= most, np.copysign(np.inf, want), want)
    bound = ref.U16[ftype] * np.abs(np.where(np.isfinite(want), want, 0)) * 1.001 + ref.TINY[ftype]
    for t in out:
        ref.check(ref.f64(t), want, bound, "read")
