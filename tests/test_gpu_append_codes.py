"""The codes and scales of the 4-bit append, byte for byte: values that are neither normed nor rotated
have right ones by their definition (dg_qkv_append in include/dg.h), whatever the factor."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from append_codes_ref import bytes_of, exact_bytes, values
from gpu_util import need_gpu
from test_gpu_head_append import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ftype", ["f16", "bf16"])
@pytest.mark.parametrize("kf,vf", [(1.0, 0.5), (0.25, 4.0), (1 / 3, 0.7), (0.1, 1.9), (3e-3, 1.1), (1e-40, 60.0)])
@pytest.mark.parametrize("heads,kvh,dim,rot,tokens,odd", [
    (2, 2, 128, 0, 40, 0), (2, 2, 64, 0, 33, 1), (1, 1, 256, 256, 20, 0), (4, 3, 96, 32, 40, 0),
    (4, 8, 128, 0, 700, 0), (12, 3, 128, 128, 700, 0), (20, 5, 64, 32, 800, 0), (9, 2, 256, 0, 560, 0),
    (17, 2, 96, 96, 560, 0),
])
def test_bytes_of_what_is_not_turned(ftype, kf, vf, heads, kvh, dim, rot, tokens, odd):
    need_gpu()
    c = Case(ftype, 4, heads, kvh, dim, 16, [1, tokens // 2, tokens - tokens // 2 - 1], seed=3, rot=rot, norm="q",
             by_map=True, kf=kf, vf=vf, odd=odd)
    c.k, c.v = values(tokens, kvh, dim, ftype, kf, 4), values(tokens, kvh, dim, ftype, vf, 5)
    edge = torch.zeros(tokens, odd, dtype=c.k.dtype)
    c.qkv = torch.cat((edge, c.q.reshape(tokens, -1), c.k.reshape(tokens, -1), c.v.reshape(tokens, -1), edge), 1)
    cache = c.run()["cache"]
    at = c.slot
    for which, x, f in ((0, c.k, kf), (1, c.v, vf)):
        if which == 0 and rot:
            continue
        nib = cache[which].numpy().reshape(-1, kvh, dim // 2)[at].astype(np.int64)
        codes = np.stack((nib & 15, nib >> 4), -1).reshape(tokens, kvh, dim)
        codes = np.where(codes > 7, codes - 16, codes)
        scales = cache[2 + which].numpy().reshape(-1, kvh, dim // 16)[at].astype(np.int64)
        want, want_s = bytes_of(ref.f64(x), f)
        assert np.array_equal(scales, want_s)
        assert np.array_equal(codes, want), (codes != want).sum()
        if np.frexp(f)[0] == 0.5:               # steps of few bits: fp32's quotients cross no border
            exact, exact_s = exact_bytes(ref.f64(x), f)
            assert np.array_equal(scales, exact_s) and np.array_equal(codes, exact)
