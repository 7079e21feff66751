"""Attention where every CTA goes through several units (sequence, head, row group), some
finished by it and some cut: each kernel variant, with several new tokens, windows and
sinks, 33 to 128 sequences, NaN in every slot that holds no position."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync
from test_gpu_attn import DT, _q, _run

pytestmark = pytest.mark.gpu
PAGE = 16


def _lens(batch, top):
    """Ragged: none, single tokens, around a block, and a few of `top`."""
    base = [0, 1, 2, 127, 128, 129, 255, 256, 257, 300, 385, top]
    return [base[i % len(base)] + (i * 7) % 40 * (i % 3 == 1) for i in range(batch)]


def _shared_pool(lens, heads, dim, dt, seed):
    """Sequences draw their pages from one pool of full pages; each one's last page is
    its own, NaN past its end."""
    g = torch.Generator().manual_seed(seed)
    shared = 64
    k, v = (torch.randn(shared + len(lens), PAGE, heads, dim, generator=g) for _ in range(2))
    width = max(-(-n // PAGE) for n in lens) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        full, rest = divmod(n, PAGE)
        table[b, :full] = torch.randint(0, shared, (full,), generator=g).int()
        k[shared + b, rest:] = v[shared + b, rest:] = float("nan")
        if rest:
            table[b, full] = shared + b
    return k.to(dt), v.to(dt), table


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 20)])
@pytest.mark.parametrize("ftype,heads,kv_heads,dim,q_len,groups,batch", [
    ("f16", 4, 2, 64, 1, 1, 100),       # 64 dims, one, two and four row tiles
    ("bf16", 4, 2, 56, 3, 1, 128),
    ("bf16", 8, 2, 64, 8, 1, 120),
    ("f16", 16, 2, 64, 7, 1, 120),
    ("bf16", 32, 2, 64, 9, 3, 45),
    ("f16", 8, 2, 128, 4, 1, 100),      # 128 dims, one and two
    ("bf16", 12, 2, 128, 5, 1, 120),
    ("f16", 24, 2, 80, 6, 3, 40),
    ("bf16", 6, 2, 192, 3, 1, 120),      # 192 and 256 dims
    ("f16", 10, 2, 160, 4, 2, 50),
    ("f16", 4, 2, 256, 2, 1, 60),
    ("bf16", 14, 2, 256, 4, 2, 40),
])
def test_many_units_a_cta(ftype, heads, kv_heads, dim, q_len, groups, batch, window, sinks):
    need_gpu()
    lens = _lens(batch, 1500)
    k, v, table = _shared_pool(lens, kv_heads, dim, DT[ftype], 90)
    table[5, 1] = -1
    ctas = torch.cuda.get_device_properties(0).multi_processor_count * (1 if dim > 192 else 2)
    seen = [min(n, window + sinks + q_len) if window else n for n in lens]
    blocks = sum(max(1, -(-n // 128)) for n in seen) * kv_heads * groups
    assert blocks > 1.2 * ctas, "the case is too small for what it tests"
    q = _q(batch * q_len, heads, dim, DT[ftype], 91)
    out, lse = _run(k, v, table, lens, q, ftype, q_len, window, sinks)
    assert torch.equal(out, _run(k, v, table, lens, q, ftype, q_len, window, sinks)[0])
    ro, rl, bo, bl = ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), table.numpy(), lens, q_len, dim ** -0.5,
                                   window, sinks, ftype)
    assert np.isfinite(ro).all()
    ref.check(ref.f64(out), ro, bo, "out")
    ref.check(ref.f64(lse), rl, bl, "lse")


@pytest.mark.parametrize("batch", [32, 33, 127, 128, 129, 300])
def test_batches_around_the_range_searches(batch):
    """Up to 32 sequences are counted by a warp, up to 128 in one pass, more in two."""
    need_gpu()
    lens = _lens(batch, 700)
    k, v, table = _shared_pool(lens, 1, 64, torch.float16, 92)
    q = _q(batch * 2, 3, 64, torch.float16, 93)
    out, lse = _run(k, v, table, lens, q, "f16", 2)
    ro, rl, bo, bl = ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), table.numpy(), lens, 2, 0.125)
    ref.check(ref.f64(out), ro, bo, "out")
    ref.check(ref.f64(lse), rl, bl, "lse")


@pytest.mark.parametrize("q_len,window,sinks", [(1, 0, 0), (3, 0, 0), (2, 100, 50), (1, 2 ** 31 - 1, 7),
                                                (2, 70, 2 ** 31 - 1)])
def test_the_longest_length(q_len, window, sinks):
    """2^31 - 1 positions, all but the last 63 in one page that the table names 2^25 - 1
    times; the last ones' page holds the strongest key.  Every position is visited where
    there is no window."""
    need_gpu()
    page, dim, n = 64, 8, 2 ** 31 - 1
    g = torch.Generator().manual_seed(94)
    k, v = (torch.randn(2, page, 1, dim, generator=g).half() for _ in range(2))
    k[0] *= 0.1
    q = torch.randn(q_len, 2, dim, generator=g).half().abs()
    k[1, 50, 0] = 30.0                                     # z >= 30 * sum(q) / sqrt(8), far above 2^31 others
    table = torch.zeros(1, 2 ** 25, dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    kd, vd, qd = k.to(DEV), v.to(DEV), q.to(DEV)
    out, lse = torch.full_like(qd, float("nan")), torch.zeros(q_len, 2, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    op = dg.attention(dg.paged_kv(kd, vd, table, lens), qd, out, lse=lse, q_len=q_len, window=window, sinks=sinks)
    ws = torch.full((dg.attn_workspace_bytes(op),), 255, dtype=torch.uint8, device=DEV)
    dg.attn_decode(op, ws)
    sync()
    z = 30.0 * ref.f64(q).sum(-1) * dim ** -0.5
    others = np.abs(ref.f64(q)).sum(-1) * np.abs(ref.f64(k[0])).max() * dim ** -0.5 + np.log(2.0 ** 31)
    near = np.abs(ref.f64(q)).sum(-1) * np.abs(ref.f64(k[1][torch.arange(page) != 50])).max() * dim ** -0.5
    assert (z > others + 9).all() and (z > near + 9).all()  # together below 63 e^-9 of the strongest
    want = ref.f64(v[1, 50, 0])
    rest = 64 * np.exp(-9.0) * (np.abs(want) + max(np.abs(ref.f64(v[0])).max(), np.abs(ref.f64(v[1])).max()))
    assert (np.abs(ref.f64(out) - want) <= rest + 2.0 ** -10 * np.abs(want)).all()
    assert (np.abs(ref.f64(lse) - z) <= 64 * np.exp(-9.0) + 1e-5 * z).all()
