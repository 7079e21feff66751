"""The 4-bit append's codes and scales of given values on the host, byte for byte.

TEST INFRASTRUCTURE ONLY.  Two forms of the definition of dg_qkv_append in include/dg.h: with quotients and
products of fp32, as the header promises them, and from products without any rounding.
"""
import numpy as np
import torch

from serve_ref import E4M3

F32 = np.float32
TABLE = E4M3[:127]                    # the scales there are, 0 to 448


def nearest_scale(q):
    """The byte of the e4m3 number nearest to q >= 0 (ties to the even byte), at most 448."""
    q = np.minimum(np.asarray(q, np.float64), 448.0)
    up = np.minimum(np.searchsorted(TABLE, q), 126)
    down = np.maximum(up - 1, 0)
    a, b = q - TABLE[down], TABLE[up] - q       # (exact: neighbours of few bits)
    return np.where(b < a, up, np.where(a < b, down, np.where(up % 2 == 0, up, down)))


def bytes_of(x, factor):
    """Codes -7..7 [.., D] and scale bytes [.., D / 16] of x [.., D], each quotient and product a number of fp32."""
    f = F32(factor)
    g = x.astype(F32).reshape(x.shape[:-1] + (-1, 16))
    top = np.abs(g).max(-1)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore", under="ignore"):
        scale = nearest_scale(top / (F32(7) * f))
        step = (TABLE.astype(F32)[scale] * f)[..., None]
        codes = np.clip(np.rint(g / step), -7, 7)
    codes = np.where(step > 0, codes, 0)
    return codes.reshape(x.shape).astype(np.int64), scale


def exact_bytes(x, factor):
    """The same from products without any rounding: s is nearest to top / (7 factor) where top lies between the
    midpoints times 7 factor, a code is above n + 1/2 where |x| is above (n + 1/2) s factor.  Products of at most 53
    bits: x of 11, s of 4, factor of 24."""
    f = float(F32(factor))
    g = x.reshape(x.shape[:-1] + (-1, 16))
    top = np.abs(g).max(-1)
    mid = (TABLE[1:] + TABLE[:-1]) / 2          # 5 significant bits
    low, high = np.searchsorted(mid * (7 * f), top, "left"), np.searchsorted(mid * (7 * f), top, "right")
    scale = np.where(low == high, low, np.where(low % 2 == 0, low, high))   # on a midpoint: the even byte
    step = (TABLE[scale] * f)[..., None]
    codes = np.zeros(g.shape, np.int64)
    for n in range(7):
        half = (n + 0.5) * step
        codes += (np.abs(g) > half) | ((np.abs(g) == half) & (n % 2 == 1))
    codes = np.where(step > 0, codes * np.sign(g).astype(np.int64), 0)
    return codes.reshape(x.shape), scale


def values(T, heads, dim, ftype, factor, seed):
    """Groups of every kind: halves of steps of all mantissas, tops at scales and halfway between two, spreads from
    below the smallest scale to past the largest."""
    r = np.random.RandomState(seed)
    x = r.randn(T, heads, dim // 16, 16) * 2.0 ** r.randint(-3, 4, (T, heads, dim // 16, 1))
    s = TABLE[r.randint(1, 127, (T, heads, dim // 16, 1))]
    halves = (r.randint(0, 7, x.shape) + 0.5) * s * r.choice([-1, 1], x.shape)
    halves[..., 3] = 7 * s[..., 0]
    middle = (TABLE[1:] + TABLE[:-1])[r.randint(1, 126, s.shape)] / 2
    between = r.uniform(-7, 7, x.shape) * middle
    between[..., 8] = -7 * middle[..., 0]
    kind = r.randint(0, 5, s.shape)
    x = np.where(kind == 1, halves, np.where(kind == 2, between, np.where(kind == 3, halves * 1e-2, x)))
    x = np.where(r.rand(*s.shape) < 0.02, x * 1000, x) * factor
    t = torch.from_numpy(x.reshape(T, heads, dim))
    top = torch.finfo(torch.float16 if ftype == "f16" else torch.bfloat16).max
    return t.clamp(-top, top).to(torch.float16 if ftype == "f16" else torch.bfloat16)
