"""The serving step's entry points on a host without a GPU: struct layouts,
workspace sizes, and every refusal before any CUDA call (fake pointers)."""
import ctypes

import pytest
import torch

import quantized_skinny_gemm_gb300 as dg

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
A, B, C, D, E, F, G, H = (0x100000 * i for i in range(1, 9))   # fake aligned addresses
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from quantized_skinny_gemm_gb300 import build
    build.build()
    return dg.load()


def _kv(**kw):
    d = dict(type=dg.F16, batch=2, kv_heads=2, head_dim=64, page_size=16, num_pages=9, max_pages=4,
             k=A, v=B, page_stride=16 * 128, token_stride=128, head_stride=64, block_table=C,
             table_stride=4, seq_lens=D)
    d.update(kw)
    return dg.PagedKV(**d)


def _kv4(**kw):
    d = dict(type=dg.F16, batch=2, kv_heads=2, head_dim=64, page_size=16, num_pages=9, max_pages=4,
             k=A, v=B, k_scale=C, v_scale=D, page_stride=16 * 64, token_stride=32, head_stride=512,
             scale_page_stride=128, scale_token_stride=4, scale_head_stride=64, k_factor=1.0, v_factor=1.0,
             block_table=E, table_stride=4, seq_lens=F)
    d.update(kw)
    return dg.PagedKV4(**d)


def _append(kv4=None, **kw):
    d = dict(kv=_kv(), kv4=kv4 or _kv4(), bits=4, q_len=1, heads=4, rot_dim=64, max_pos=100, eps=1e-6, q=A, k=B, v=C,
             q_out=D, q_stride=256, k_stride=128, v_stride=128, q_out_stride=256, cos=A, sin=B, w_q=C, w_k=D)
    d.update(kw)
    return dg.HeadAppend(**d)


def _rows(kv=None, **kw):
    d = dict(kv=kv or _kv4(), q_len=3, tokens=6, k=A, v=B, k_stride=128, v_stride=128)
    d.update(kw)
    return dg.KV4Rows(**d)


def _attn(kv=None, **kw):
    d = dict(kv=kv or _kv4(), q_len=1, heads=4, scale=0.125, q=A, out=B, q_stride=256, out_stride=256)
    d.update(kw)
    return dg.Attention4(**d)


def _plan(**kw):
    d = dict(batch=3, page_size=16, max_pages=4, pool_size=20, new_len=1, max_tokens=8, table_stride=4, lens=A,
             new_lens=B, lens_out=C, block_table=D, pool=E, pool_state=F, pool_state_out=G, starts=H, slots=H + 4096,
             positions=H + 8192)
    d.update(kw)
    return dg.PagePlan(**d)


def _logprobs(**kw):
    d = dict(type=dg.F16, logits_f32=1, rows=3, V=100, top_k=5, scale=1.0, stride=100, logits=A, tokens=B, logprob=C,
             rank=D, entropy=E, lse=F, top_ids=G, top_logprobs=H)
    d.update(kw)
    return dg.Logprobs(**d)


def test_struct_layouts():
    size = ctypes.sizeof
    assert size(dg.PagedKV4) == 144 and dg.PagedKV4.k.offset == 32 and dg.PagedKV4.k_factor.offset == 112
    assert dg.PagedKV4.seq_lens.offset == 136
    assert size(dg.HeadAppend) == 392 and dg.HeadAppend.kv4.offset == 96 and dg.HeadAppend.bits.offset == 240
    assert dg.HeadAppend.q.offset == 280 and dg.HeadAppend.positions.offset == 384
    assert size(dg.KV4Rows) == 192 and dg.KV4Rows.k.offset == 152
    assert size(dg.Attention4) == 208 and dg.Attention4.scale.offset == 160 and dg.Attention4.q.offset == 168
    assert size(dg.PagePlan) == 112 and dg.PagePlan.lens.offset == 32
    assert size(dg.Logprobs) == 96 and dg.Logprobs.logits.offset == 32


def test_cache_refusals(lib):
    def every(kv):
        got = {lib.dg_attn4_decode(ctypes.byref(_attn(kv)), A, 1 << 30, None),
               lib.dg_qkv_append(ctypes.byref(_append(kv)), None),
               lib.dg_kv4_read(ctypes.byref(_rows(kv, tokens=3 * max(kv.batch, 1))), None)}
        assert lib.dg_attn4_workspace_bytes(ctypes.byref(_attn(kv))) == 0
        assert len(got) == 1
        return got.pop()
    for bad in (dict(type=2), dict(batch=0), dict(kv_heads=0), dict(head_dim=0), dict(page_size=0),
                dict(num_pages=0), dict(max_pages=0), dict(reserved=1), dict(k=None), dict(v=None),
                dict(k_scale=None), dict(v_scale=None), dict(block_table=None), dict(seq_lens=None),
                dict(page_stride=-8), dict(token_stride=-8), dict(head_stride=-8), dict(scale_page_stride=-1),
                dict(scale_token_stride=-1), dict(scale_head_stride=-1), dict(table_stride=3),
                dict(k_factor=0.0), dict(v_factor=0.0), dict(k_factor=-1.0), dict(v_factor=NAN),
                dict(k_factor=INF), dict(v_factor=INF), dict(k_factor=1e38), dict(v_factor=1e38)):
        assert every(_kv4(**bad)) == INVALID, bad
    for bad in (dict(head_dim=24), dict(head_dim=8), dict(head_dim=272), dict(batch=(1 << 20) + 1), dict(kv_heads=2048),
                dict(page_stride=1 << 32), dict(token_stride=1 << 32), dict(head_stride=1 << 40),
                dict(scale_page_stride=1 << 32), dict(scale_token_stride=1 << 32), dict(scale_head_stride=1 << 32)):
        assert every(_kv4(**bad)) == UNSUPPORTED, bad
    for bad in (dict(block_table=E + 2), dict(seq_lens=F + 2), dict(k=A + 4), dict(v=B + 4), dict(page_stride=1028),
                dict(token_stride=36), dict(head_stride=516)):
        assert every(_kv4(**bad)) == MISALIGNED, bad


def test_append_refusals(lib):
    f = lambda **kw: lib.dg_qkv_append(ctypes.byref(_append(**kw)), None)
    assert lib.dg_qkv_append(None, None) == INVALID
    for bad in (dict(bits=8), dict(q_len=0), dict(tokens=1), dict(positions=A), dict(heads=-1), dict(q=None),
                dict(q_out=None), dict(heads=0), dict(k=None), dict(v=None), dict(interleaved=2), dict(rot_dim=-2),
                dict(rot_dim=3), dict(rot_dim=66), dict(cos=None), dict(sin=None), dict(max_pos=0),
                dict(q_stride=-1), dict(k_stride=-1), dict(v_stride=-1), dict(q_out_stride=255),
                dict(q_out=A, q_out_stride=512), dict(norm=2), dict(eps=-1.0), dict(eps=NAN), dict(w_offset=INF),
                dict(heads=0, q=None, q_out=None),                      # w_q without q
                dict(slots=A, q_len=0, tokens=5), dict(slots=A, positions=B, q_len=0, tokens=0),
                dict(slots=A, positions=B, q_len=1, tokens=5)):
        assert f(**bad) == INVALID, bad
    assert f(q_len=17) == UNSUPPORTED and f(heads=2000) == UNSUPPORTED
    assert f(slots=A, positions=B, q_len=0, tokens=2 ** 31 - 1) == UNSUPPORTED
    for bad in (dict(q=A + 1), dict(k=A + 1), dict(v=A + 1), dict(q_out=A + 1), dict(w_q=A + 1), dict(w_k=A + 1),
                dict(cos=A + 2), dict(sin=A + 2), dict(slots=A + 4, positions=B, q_len=0, tokens=5),
                dict(slots=A, positions=B + 2, q_len=0, tokens=5), dict(bits=16, kv=_kv(k=A + 1))):
        assert f(**bad) == MISALIGNED, bad
    assert f(bits=16, kv=_kv(head_dim=0)) == INVALID and f(bits=16, kv=_kv(head_dim=12)) == UNSUPPORTED
    # the cache that is not meant is not looked at
    assert f(bits=16, kv=_kv(type=7)) == INVALID and f(bits=4, kv=_kv(type=7), k=None) == INVALID


def test_read_refusals(lib):
    f = lambda **kw: lib.dg_kv4_read(ctypes.byref(_rows(**kw)), None)
    assert lib.dg_kv4_read(None, None) == INVALID
    for bad in (dict(tokens=0), dict(tokens=5), dict(q_len=0), dict(k=None, v=None), dict(k_stride=127),
                dict(v_stride=64), dict(slots=A), dict(slots=A, q_len=0, tokens=0)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(k=A + 1), dict(v=A + 1), dict(slots=A + 4, q_len=0)):
        assert f(**bad) == MISALIGNED, bad


def test_attention_refusals(lib):
    f = lambda ws=A, n=1 << 30, **kw: lib.dg_attn4_decode(ctypes.byref(_attn(**kw)), ws, n, None)
    assert lib.dg_attn4_decode(None, A, 1 << 30, None) == INVALID
    for bad in (dict(q_len=0), dict(heads=0), dict(heads=5), dict(q=None), dict(out=None), dict(window=-1),
                dict(sinks=-1), dict(scale=NAN), dict(scale=INF), dict(scale=2e37), dict(reserved=1),
                dict(q_stride=-8), dict(out_stride=248), dict(scale=1e20, kv=_kv4(k_factor=1e20))):
        assert f(**bad) == INVALID, bad
    assert f(q_len=17) == UNSUPPORTED
    assert f(heads=2050) == UNSUPPORTED
    for bad in (dict(q=A + 8), dict(out=B + 8), dict(q_stride=260), dict(out_stride=260), dict(lse=A + 2)):
        assert f(**bad) == MISALIGNED, bad
    need = lib.dg_attn4_workspace_bytes(ctypes.byref(_attn(_kv4(max_pages=40, table_stride=40))))
    assert need > lib.dg_attn4_workspace_bytes(ctypes.byref(_attn())) > 0
    big = dict(kv=_kv4(max_pages=40, table_stride=40))
    assert f(ws=None, **big) == WORKSPACE and f(n=need - 1, **big) == WORKSPACE
    assert f(ws=A + 8, n=need, **big) == MISALIGNED


def test_page_refusals(lib):
    f = lambda ws=A + 0x900000, n=1 << 30, **kw: lib.dg_assign_pages(ctypes.byref(_plan(**kw)), ws, n, None)
    assert lib.dg_assign_pages(None, A, 1 << 30, None) == INVALID
    for bad in (dict(batch=0), dict(page_size=0), dict(max_pages=0), dict(pool_size=0), dict(max_tokens=-1),
                dict(lens=None), dict(lens_out=None), dict(block_table=None), dict(pool=None), dict(pool_state=None),
                dict(pool_state_out=None), dict(slots=None), dict(max_tokens=0), dict(slots=None, max_tokens=0),
                dict(table_stride=3),
                # overlapping memory
                dict(lens_out=A + 4), dict(lens_out=B), dict(block_table=A), dict(pool=D + 44), dict(pool=F - 4),
                dict(pool_state_out=F + 4), dict(starts=A + 8), dict(slots=H + 8), dict(positions=H + 4096 + 60),
                dict(lens=C, lens_out=C, new_lens=C), dict(starts=G)):
        assert f(**bad) == INVALID, bad
    assert f(batch=(1 << 20) + 1) == UNSUPPORTED
    for bad in (dict(lens=A + 2), dict(new_lens=B + 2), dict(lens_out=C + 2), dict(block_table=D + 2),
                dict(pool=E + 2), dict(pool_state=F + 2), dict(starts=H + 2), dict(slots=H + 4100),
                dict(positions=H + 8194)):
        assert f(**bad) == MISALIGNED, bad
    size = lambda **kw: lib.dg_pages_workspace_bytes(ctypes.byref(_plan(**kw)))
    far = dict(lens=0x10000000, new_lens=0x20000000, lens_out=0x30000000, block_table=0x40000000, pool=0x50000000,
               starts=0x60000000, slots=0x70000000, positions=0x80000000)
    assert size() == 0 and size(batch=0) == 0
    many = dict(far, batch=5000)
    need = size(**many)
    assert need >= 5000 * 16 and size(**dict(far, max_tokens=1 << 20)) > 0
    assert f(ws=None, **many) == WORKSPACE and f(n=need - 1, **many) == WORKSPACE
    assert f(ws=A + 8, n=need, **many) == MISALIGNED


def test_logprob_refusals(lib):
    f = lambda ws=A, n=1 << 30, **kw: lib.dg_token_logprobs(ctypes.byref(_logprobs(**kw)), ws, n, None)
    assert lib.dg_token_logprobs(None, A, 1 << 30, None) == INVALID
    for bad in (dict(type=2), dict(logits_f32=2), dict(rows=0), dict(V=0), dict(top_k=-1), dict(V=4, stride=4),
                dict(logits=None), dict(stride=99), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
                dict(scale=INF), dict(scale=3e38), dict(tokens=None), dict(tokens=None, logprob=None),
                dict(top_k=0), dict(top_ids=None, top_logprobs=None),
                dict(top_k=0, top_ids=None, top_logprobs=None, logprob=None, rank=None, entropy=None, lse=None)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(top_k=33), dict(rows=(1 << 22) + 1), dict(V=(1 << 30) + 1, stride=1 << 31)):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(logits=A + 2), dict(logits_f32=0, logits=A + 1), dict(tokens=B + 2), dict(logprob=C + 2),
                dict(rank=D + 1), dict(entropy=E + 2), dict(lse=F + 2), dict(top_ids=G + 2), dict(top_logprobs=H + 2)):
        assert f(**bad) == MISALIGNED, bad
    big = dict(V=200000, stride=200000)
    need = lib.dg_logprobs_workspace_bytes(ctypes.byref(_logprobs(**big)))
    assert need > 0 and lib.dg_logprobs_workspace_bytes(ctypes.byref(_logprobs(**dict(big, rows=0)))) == 0
    assert f(ws=None, **big) == WORKSPACE and f(n=need - 1, **big) == WORKSPACE
    assert f(ws=A + 8, n=need, **big) == MISALIGNED
    assert lib.dg_logprobs_workspace_bytes(ctypes.byref(_logprobs(rows=4000))) == 0


def test_builders_refuse_tensors_that_do_not_fit():
    t, i32, f16 = torch.zeros, torch.int32, torch.float16
    u8 = lambda *s: t(*s, dtype=torch.uint8)
    table, lens = t(2, 4, dtype=i32), t(2, dtype=i32)
    codes, scales = u8(9, 16, 2, 32), u8(9, 16, 2, 4)
    kv = dg.paged_kv4(codes, codes, scales, scales.view(torch.float8_e4m3fn).view(torch.uint8), table, lens)
    assert (kv.head_dim, kv.batch, kv.num_pages, kv.max_pages, kv.type) == (64, 2, 9, 4, dg.F16)
    swapped = dg.paged_kv4(u8(9, 2, 16, 32).transpose(1, 2), u8(9, 2, 16, 32).transpose(1, 2),
                           u8(9, 2, 16, 4).transpose(1, 2), u8(9, 2, 16, 4).transpose(1, 2), table, lens,
                           dtype=torch.bfloat16)
    assert (swapped.token_stride, swapped.head_stride, swapped.scale_head_stride) == (32, 512, 64)

    def refused(f):
        with pytest.raises(dg.DGError):
            f()
    refused(lambda: dg.paged_kv4(codes, u8(9, 16, 2, 40), scales, scales, table, lens))
    refused(lambda: dg.paged_kv4(codes, codes, u8(9, 16, 2, 2), u8(9, 16, 2, 2), table, lens))
    refused(lambda: dg.paged_kv4(codes.char(), codes.char(), scales, scales, table, lens))
    refused(lambda: dg.paged_kv4(codes, codes, scales, scales, table.long(), lens))
    refused(lambda: dg.paged_kv4(codes, codes, scales, scales, table[:1].expand(2, 4), lens))
    refused(lambda: dg.paged_kv4(codes, codes, scales, scales, table, lens, dtype=torch.float32))
    q, k = t(2, 4, 64, dtype=f16), t(2, 2, 64, dtype=f16)
    assert dg.head_append(kv, q, k, k).tokens == 0
    slots, pos = t(5, dtype=torch.int64), t(5, dtype=i32)
    five = t(5, 2, 64, dtype=f16)
    assert dg.head_append(kv, None, five, five, slots=slots, positions=pos).tokens == 5
    refused(lambda: dg.head_append(kv, q, five, k))
    refused(lambda: dg.head_append(kv, q, k.bfloat16(), k))
    refused(lambda: dg.head_append(kv, q, k, k, w_q=t(63, dtype=f16)))
    refused(lambda: dg.head_append(kv, q, k, k, w_q=t(64)))
    refused(lambda: dg.head_append(kv, None, five, five, slots=slots))
    refused(lambda: dg.head_append(kv, None, five, five, slots=slots, positions=pos, q_len=1))
    refused(lambda: dg.head_append(kv, None, five, five, slots=slots, positions=pos[:4]))
    refused(lambda: dg.head_append(kv, q, k, k, cos=t(9, 32)))
    refused(lambda: dg.kv4_rows(kv, None, None))
    refused(lambda: dg.kv4_rows(kv, five))
    refused(lambda: dg.kv4_rows(kv, k[:1].expand(2, 2, 64)))          # rows over each other
    assert dg.kv4_rows(kv, k).k_stride == 128
    refused(lambda: dg.attention4(kv, q, t(2, 4, 32, dtype=f16)))
    refused(lambda: dg.attention4(kv, q.bfloat16(), q.bfloat16()))
    pool, state = t(20, dtype=i32), t(2, dtype=i32)
    assert dg.page_plan(lens, table, pool, state, 16).max_tokens == 0
    refused(lambda: dg.page_plan(lens, table, pool, state[:1], 16))
    refused(lambda: dg.page_plan(lens, table, pool, state, 16, new_lens=t(3, dtype=i32)))
    refused(lambda: dg.page_plan(lens, table, pool, state, 16, slots=slots, positions=pos[:3]))
    refused(lambda: dg.page_plan(lens, table, pool, state, 16, slots=pos))
    x, one = t(3, 100), t(3)
    assert dg.logprobs(x, entropy=one).stride == 100 and dg.logprobs(x[0], entropy=one[:1]).rows == 1
    refused(lambda: dg.logprobs(x.double(), entropy=one))
    refused(lambda: dg.logprobs(x, entropy=t(2)))
    refused(lambda: dg.logprobs(x.t(), entropy=t(100)))
    refused(lambda: dg.logprobs(x, tokens=t(3, dtype=torch.int64), logprob=one))
    refused(lambda: dg.logprobs(x, top_ids=t(3, 4, dtype=i32), top_logprobs=t(3, 5)))


def test_builders_refuse_sizes_past_32_bits():
    """A count of 2^32 + 5 is not one of 5."""
    big = 2 ** 32 + 5
    meta = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="meta")
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    with pytest.raises(dg.DGError):
        dg.page_plan(i32(2), i32(2, 4), i32(8), i32(2), 16, slots=meta(big, dtype=torch.int64))
    with pytest.raises(dg.DGError):
        dg.page_plan(i32(2), i32(2, 4), meta(big), i32(2), 16)
    with pytest.raises(dg.DGError):
        dg.logprobs(meta(big, 4, dtype=torch.float16), lse=meta(big, dtype=torch.float32))
    with pytest.raises(dg.DGError):
        dg.logprobs(meta(1, big, dtype=torch.float16), lse=meta(1, dtype=torch.float32))
    codes = lambda w: torch.zeros(4, 16, 1, w, dtype=torch.uint8)
    kv = dg.paged_kv4(codes(8), codes(8), codes(1), codes(1), i32(2, 4), i32(2))
    half = lambda: meta(big, 1, 16, dtype=torch.float16)
    slots = meta(big, dtype=torch.int64)
    with pytest.raises(dg.DGError):
        dg.kv4_rows(kv, half(), slots=slots)
    with pytest.raises(dg.DGError):
        dg.head_append(kv, None, half(), half(), slots=slots, positions=meta(big))


def test_only_lengths_and_state_may_be_their_own_outputs(lib):
    f = lambda **kw: lib.dg_assign_pages(ctypes.byref(_plan(**kw)), A + 0x900000, 1 << 30, None)
    for at in (D, C, E, G, H, H + 4096, H + 8192):      # what is written
        assert f(new_lens=at) == INVALID
    assert f(lens=G, lens_out=C, pool_state_out=G) == INVALID and f(pool_state=C, lens_out=C) == INVALID


def test_builders_refuse_whole_numbers_past_32_bits():
    """A page of 2^32 + 16 positions is not one of 16, a window of 2^32 not none."""
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    f16 = lambda *shape: torch.zeros(shape, dtype=torch.float16)
    codes = lambda w: torch.zeros(4, 16, 1, w, dtype=torch.uint8)
    kv = dg.paged_kv4(codes(8), codes(8), codes(1), codes(1), i32(2, 4), i32(2))
    plan = lambda page=16, **kw: dg.page_plan(i32(2), i32(2, 4), i32(8), i32(2), page, **kw)
    attn = lambda **kw: dg.attention4(kv, f16(2, 1, 16), f16(2, 1, 16), **kw)
    assert plan(new_len=-2 ** 31).new_len == -2 ** 31 and plan(2 ** 31 - 1).page_size == 2 ** 31 - 1
    assert attn(window=2 ** 31 - 1, sinks=2 ** 31 - 1).window == 2 ** 31 - 1
    for build in (lambda: plan(2 ** 32 + 16), lambda: plan(2 ** 31), lambda: plan(new_len=2 ** 32 + 1),
                  lambda: plan(new_len=-2 ** 32), lambda: attn(window=2 ** 32), lambda: attn(window=2 ** 32 + 100),
                  lambda: attn(sinks=2 ** 32 + 4), lambda: attn(sinks=-2 ** 32)):
        with pytest.raises(dg.DGError):
            build()
