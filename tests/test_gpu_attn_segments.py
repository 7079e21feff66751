"""Attention where every CTA goes through several units (sequence, head, row group), some
finished by it and some cut: each kernel variant, with several new tokens, windows and
sinks, 33 to 128 sequences, NaN in every slot that holds no position."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from gpu_util import need_gpu
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
    ("bf16", 12, 2, 256, 4, 2, 40),
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
