"""The decoder-layer entry points on a host without a GPU: struct layouts,
workspace sizes, and every refusal before any CUDA call (fake pointers)."""
import ctypes

import pytest
import torch

import quantized_skinny_gemm_gb300 as dg
from quantized_skinny_gemm_gb300 import plans, synth

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000   # fake aligned addresses
ODD = 0x100008


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


def _attn(kv=None, **kw):
    d = dict(kv=kv or _kv(), q_len=1, heads=4, scale=0.125, q=A, out=B, q_stride=256, out_stride=256)
    d.update(kw)
    return dg.Attention(**d)


def _append(kv=None, **kw):
    d = dict(kv=kv or _kv(), q_len=1, heads=4, rot_dim=64, max_pos=100, q=A, k=B, v=C, q_out=D,
             q_stride=256, k_stride=128, v_stride=128, q_out_stride=256, cos=A, sin=B)
    d.update(kw)
    return dg.Append(**d)


def _norm(**kw):
    d = dict(type=dg.F16, rows=2, N=64, alpha=1.0, beta=1.0, eps=1e-6, y=A, h=B, w_pre=C, h_out=D,
             x_out=D + 0x10000)
    d.update(kw)
    return dg.Norm(**d)


def _moe(**kw):
    d = dict(kind=dg.LINEAR_F16, M=1, K=64, I=64, E=8, top_k=2, route_scale=1.0, x=A, router=A, W_gate=A,
             W_up=A, W_down=A, y=B)
    d.update(kw)
    return dg.Moe(**d)


def test_struct_layouts():
    assert ctypes.sizeof(dg.PagedKV) == 96 and dg.PagedKV.k.offset == 32
    assert dg.PagedKV.seq_lens.offset == 88
    assert ctypes.sizeof(dg.Append) == 96 + 24 + 80 and dg.Append.q.offset == 120
    assert ctypes.sizeof(dg.Attention) == 96 + 24 + 40 and dg.Attention.scale.offset == 112
    assert ctypes.sizeof(dg.Norm) == 40 + 72 and dg.Norm.y.offset == 40
    assert ctypes.sizeof(dg.Moe) == 40 + 96 and dg.Moe.x.offset == 40


def test_cache_refusals(lib):
    def both(kv):
        a = lib.dg_attn_decode(ctypes.byref(_attn(kv)), A, 1 << 30, None)
        b = lib.dg_kv_append(ctypes.byref(_append(kv)), None)
        assert a == b
        assert lib.dg_attn_workspace_bytes(ctypes.byref(_attn(kv))) == 0
        return a
    for bad in (dict(type=2), dict(batch=0), dict(kv_heads=0), dict(head_dim=0), dict(page_size=0),
                dict(num_pages=0), dict(max_pages=0), dict(reserved=1), dict(k=None), dict(v=None),
                dict(block_table=None), dict(seq_lens=None), dict(page_stride=-8), dict(token_stride=-8),
                dict(head_stride=-8), dict(table_stride=3)):
        assert both(_kv(**bad)) == INVALID, bad
    for bad in (dict(head_dim=12), dict(head_dim=264), dict(batch=(1 << 20) + 1), dict(kv_heads=2048)):
        assert both(_kv(**bad)) == UNSUPPORTED, bad
    for bad in (dict(block_table=C + 2), dict(seq_lens=D + 2)):
        assert both(_kv(**bad)) == MISALIGNED, bad


def test_attention_refusals(lib):
    f = lambda ws=A, n=1 << 30, **kw: lib.dg_attn_decode(ctypes.byref(_attn(**kw)), ws, n, None)
    assert lib.dg_attn_decode(None, A, 1 << 30, None) == INVALID
    for bad in (dict(q_len=0), dict(heads=0), dict(heads=5), dict(q=None), dict(out=None), dict(window=-1),
                dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(reserved=1),
                dict(q_stride=-8), dict(out_stride=248)):
        assert f(**bad) == INVALID, bad
    assert f(q_len=17) == UNSUPPORTED
    assert f(heads=2050) == UNSUPPORTED
    for bad in (dict(q=ODD), dict(out=ODD), dict(q_stride=260), dict(out_stride=260), dict(lse=A + 2),
                dict(kv=_kv(k=ODD)), dict(kv=_kv(v=ODD)), dict(kv=_kv(page_stride=2052)),
                dict(kv=_kv(token_stride=132)), dict(kv=_kv(head_stride=68))):
        assert f(**bad) == MISALIGNED, bad
    need = lib.dg_attn_workspace_bytes(ctypes.byref(_attn()))
    assert need > 0
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE
    assert f(ws=ODD, n=need) == MISALIGNED


def test_append_refusals(lib):
    f = lambda **kw: lib.dg_kv_append(ctypes.byref(_append(**kw)), None)
    assert lib.dg_kv_append(None, None) == INVALID
    for bad in (dict(heads=-1), dict(q=None), dict(q_out=None), dict(heads=0), dict(k=None), dict(v=None),
                dict(interleaved=2), dict(rot_dim=-2), dict(rot_dim=3), dict(rot_dim=66), dict(cos=None),
                dict(sin=None), dict(max_pos=0), dict(q_stride=-1), dict(k_stride=-1), dict(v_stride=-1),
                dict(q_out_stride=255), dict(q_out=A, q_out_stride=512), dict(reserved=1)):
        assert f(**bad) == INVALID, bad
    assert f(q_len=17) == UNSUPPORTED
    for bad in (dict(q=A + 1), dict(k=A + 1), dict(cos=A + 2), dict(sin=A + 2)):
        assert f(**bad) == MISALIGNED, bad


def test_norm_refusals(lib):
    f = lambda **kw: lib.dg_norm_residual(ctypes.byref(_norm(**kw)), None)
    assert lib.dg_norm_residual(None, None) == INVALID
    for bad in (dict(type=2), dict(kind=2), dict(rows=0), dict(N=0), dict(h_f32=2), dict(y=None, h=None),
                dict(y=None, w_post=A), dict(y=None, gate=A, gate_rows=1), dict(b_post=A), dict(w_pre=None),
                dict(x_out=None, w_pre=None, b_pre=A), dict(h_out=None, x_out=None), dict(gate_rows=1),
                dict(gate=A + 0x50000, gate_rows=3), dict(eps=-1e-6), dict(eps=float("nan")),
                dict(alpha=float("inf")), dict(beta=float("nan")), dict(w_offset=float("inf"))):
        assert f(**bad) == INVALID, bad
    for bad in (dict(h_out=B + 16), dict(h_out=C), dict(x_out=D), dict(x_out=D + 16),
                dict(h_f32=1, h_out=A), dict(h_f32=1, x_out=B)):     # overlapping memory
        assert f(**bad) == INVALID, bad
    assert f(N=32769) == UNSUPPORTED
    for bad in (dict(h=B + 1), dict(h_f32=1, h=B + 2), dict(w_pre=C + 1), dict(y=A + 1)):
        assert f(**bad) == MISALIGNED, bad


def test_moe_refusals(lib):
    f = lambda ws=A, n=1 << 30, **kw: lib.dg_moe_forward(ctypes.byref(_moe(**kw)), ws, n, None)
    w4 = dict(kind=dg.LINEAR_W4A16, group_size=32, gate_scale=A, up_scale=A, down_scale=A)
    assert lib.dg_moe_forward(None, A, 1 << 30, None) == INVALID
    for bad in (dict(kind=-1), dict(kind=7), dict(M=0), dict(K=0), dict(I=0), dict(E=0), dict(top_k=0),
                dict(top_k=9), dict(score=2), dict(renormalize=2), dict(route_scale=float("nan")),
                dict(x=None), dict(router=None), dict(W_gate=None), dict(W_up=None), dict(W_down=None),
                dict(y=None), dict(w4, gate_scale=None), dict(w4, down_scale=None)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(kind=dg.LINEAR_W8A8), dict(kind=dg.LINEAR_W4A8), dict(M=17), dict(E=1025),
                dict(E=64, top_k=17), dict(K=65544), dict(I=65544), dict(w4, group_size=48),
                dict(w4, group_size=16), dict(w4, K=96, group_size=64)):
        assert f(**bad) == UNSUPPORTED, bad
    for bad in (dict(K=60), dict(I=68), dict(x=ODD), dict(y=ODD), dict(W_down=ODD), dict(residual=A + 1),
                dict(ids=A + 2), dict(weights=A + 2), dict(w4, up_scale=A + 1)):
        assert f(**bad) == MISALIGNED, bad
    need = lib.dg_moe_workspace_bytes(ctypes.byref(_moe()))
    assert need > 0 and lib.dg_moe_workspace_bytes(ctypes.byref(_moe(M=17))) == 0
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE
    assert f(ws=ODD, n=need) == MISALIGNED


def test_builders_refuse_tensors_that_do_not_fit():
    h = lambda *s, dt=torch.float16: torch.zeros(*s, dtype=dt)
    k, table, lens = h(4, 16, 2, 64), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kv = dg.paged_kv(k, k.clone(), table, lens)
    assert (kv.page_stride, kv.token_stride, kv.head_stride, kv.max_pages) == (2048, 128, 64, 3)
    turned = k.view(4, 2, 16, 64).transpose(1, 2)
    assert dg.paged_kv(turned, turned, table, lens).head_stride == 16 * 64
    for bad in ((k, k.transpose(1, 2).contiguous().transpose(1, 2), table, lens),
                (k, h(4, 16, 2, 32), table, lens), (k.float(), k.float(), table, lens),
                (k, k, table.long(), lens), (k, k, table, lens[:1])):
        with pytest.raises(dg.DGError):
            dg.paged_kv(*bad)
    q = h(2, 4, 64)
    op = dg.attention(kv, q, q.clone())
    assert op.heads == 4 and op.q_stride == 256 and abs(op.scale - 0.125) < 1e-9
    for kw in (dict(q=q.bfloat16(), out=q), dict(q=q, out=h(2, 3, 64)), dict(q=q, out=q, q_len=0),
               dict(q=q, out=q, lse=h(2, 4)), dict(q=h(2, 4, 128)[..., :64].transpose(1, 2), out=q)):
        with pytest.raises(dg.DGError):
            dg.attention(kv, **kw)
    with pytest.raises(dg.DGError):
        dg.append(kv, q, h(2, 2, 64), h(2, 3, 64))
    with pytest.raises(dg.DGError):
        dg.append(kv, q, h(2, 2, 64), h(2, 2, 64), cos=torch.zeros(9, 32), sin=torch.zeros(9, 16))
    with pytest.raises(dg.DGError):
        dg.norm(h(2, 8), h(2, 8), h(2, 8), w_pre=h(9))
    with pytest.raises(dg.DGError):
        dg.norm(h(2, 8).float(), h(2, 8), h(2, 8), w_pre=h(8))
    with pytest.raises(dg.DGError):
        dg.moe(dg.LINEAR_F16, h(1, 64), h(1, 64), h(4, 64), h(4, 32, 64), h(4, 32, 64), h(4, 64, 40), 2)


def test_a_page_table_is_described_with_its_own_stride():
    """Rows that overlap are refused: sequences would read past the table."""
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    ids = torch.zeros(64, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    for rows, stride in ((2, 3), (2, 5), (1, 0), (1, 1)):
        kv = dg.paged_kv(k, k, ids.as_strided((rows, 3), (stride, 1)), lens[:rows])
        assert kv.max_pages == 3 and kv.table_stride == (stride if rows > 1 else 3)
    assert dg.paged_kv(k, k, ids.as_strided((2, 1), (4, 9)), lens).table_stride == 4
    for table in (ids[:3].expand(2, 3), ids.as_strided((2, 3), (1, 1)), ids.as_strided((2, 3), (2, 1)),
                  ids[:1].expand(2, 1)):
        with pytest.raises(dg.DGError):
            dg.paged_kv(k, k, table, lens)


def test_scales_that_overflow_are_refused(lib):
    """Scores are held in units of log2(e)."""
    f = lambda scale: lib.dg_attn_decode(ctypes.byref(_attn(scale=scale)), A, 0, None)
    for scale in (2.5e38, -3.4e38):
        assert f(scale) == INVALID
    for scale in (2.3e38, -2.3e38, 0.0, 1e-45, -1e-39):
        assert f(scale) == WORKSPACE      # taken, and refused for its workspace


def test_a_sparse_plan_refuses_what_its_operators_would(lib):
    """At the plan, not at run() behind the first norm."""
    layers = synth.sparse_decoder_workload(1, 1, 64, 4, 2, 16, 32, 4)
    plan = lambda heads=4, kv_heads=2, top_k=2, **kw: plans.sparse_decoder_step(
        layers, torch.device("cpu"), heads, kv_heads, top_k, max_pages=2, **kw)
    for kw in (dict(), dict(batch=4, q_len=4), dict(q_len=16), dict(batch=16), dict(window=9, sinks=2)):
        step = plan(**kw)
        assert step.h.shape == (kw.get("batch", 1) * kw.get("q_len", 1), 64)
    for kw in (dict(batch=17), dict(q_len=17), dict(batch=3, q_len=6), dict(batch=0), dict(q_len=0), dict(top_k=5),
               dict(window=-1), dict(heads=8)):
        with pytest.raises((ValueError, dg.DGError)):
            plan(**kw)


def test_a_gate_of_one_value_a_row_is_refused():
    """[rows][1] has as many values as a row [N] where rows == N."""
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    op = lambda gate, rows=8: dg.norm(h(rows, 8), h(rows, 8), None, y=h(rows, 8), gate=gate)
    assert op(h(8)).gate_rows == 1 and op(h(1, 8)).gate_rows == 1 and op(h(8, 8)).gate_rows == 8
    assert op(h(64)).gate_rows == 8 and op(h(4, 2, 8)).gate_rows == 8
    for gate in (h(8, 1), h(2, 4), h(16, 4), h(8, 8, 1)):
        with pytest.raises(dg.DGError):
            op(gate)


def test_half_a_rotation_is_refused():
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    kv = dg.paged_kv(h(4, 16, 2, 64), h(4, 16, 2, 64), torch.zeros(2, 3, dtype=torch.int32),
                     torch.zeros(2, dtype=torch.int32))
    table = torch.zeros(9, 32)
    op = lambda **kw: dg.append(kv, h(2, 4, 64), h(2, 2, 64), h(2, 2, 64), **kw)
    assert op(cos=table, sin=table).rot_dim == 64 and op().rot_dim == 0
    for kw in (dict(sin=table), dict(cos=table)):
        with pytest.raises(dg.DGError):
            op(**kw)
