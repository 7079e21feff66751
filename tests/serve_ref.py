"""The serving step's operators in 64 bits, with error bounds.

TEST INFRASTRUCTURE ONLY.  numpy float64 and whole numbers on the host, from the
definitions in include/dg.h; the bounds follow the arithmetic that the header
promises, as in layer_ref (fp32 sums, one rounding into the output).
"""
import numpy as np

import layer_ref as ref
from layer_ref import FN, TINY, U16, U32


def e4m3_values():
    """The 256 values of e4m3 (fn: no infinities, 0x7F and 0xFF are NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where(b & 127 == 127, np.nan, v)
    return np.where(b > 127, -v, v)


E4M3 = e4m3_values()


def decode4(codes, scales, factor):
    """codes uint8 [.., D / 2], scales uint8 [.., D / 16] -> float64 [.., D]."""
    lo, hi = (codes & 15).astype(np.int64), (codes >> 4).astype(np.int64)
    c = np.stack((lo, hi), -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    c = np.where(c > 7, c - 16, c).astype(np.float64)
    return c * np.repeat(E4M3[scales], 16, axis=-1) * factor


def attention4(q, k, v, table, lens, q_len, scale, window=0, sinks=0, ftype="f16"):
    """As layer_ref.attention over a decoded cache, with the bounds of dg_attn4_decode: a
    score errs by D fp32 roundings of its products and a few of itself; a weight by
    that, its function, and 2^-21 as two fp16 numbers, or 2^-32 of the strongest
    key's; bf16 queries lose what lies below 2^-30 of their row's largest."""
    T, H, D = q.shape
    P, S, G, _ = k.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    b_out, b_lse = np.full((T, H, D), TINY[ftype]), np.zeros((T, H))
    table = np.where((table >= 0) & (table < P), table, -1)
    for t in range(T):
        b = t // q_len
        p = int(lens[b]) - q_len + t % q_len
        j = ref.visible(p, table.shape[1] * S, table[b], S, window, sinks)
        if not j.size:
            continue
        pg, sl = table[b][j // S], j % S
        for h in range(H):
            kk, vv = k[pg, sl, h // (H // G)], v[pg, sl, h // (H // G)]
            with np.errstate(invalid="ignore", over="ignore"):
                z = scale * (kk @ q[t, h])
                m = z.max()
                if m == -np.inf:
                    continue
                e = np.exp(z - m)
                l = e.sum()
                out[t, h] = e @ vv / l
                lse[t, h] = m + np.log(l)
                lost = (np.abs(kk).sum(1) * np.abs(q[t, h]).max() * 2.0 ** -30 if ftype == "bf16" else 0.0)
                ez = (abs(scale) * ((D + 2) * U32 * (np.abs(kk) @ np.abs(q[t, h])) + lost)
                      + 4 * U32 * (np.abs(z) + abs(m)))
                rel = ez.max() + FN + (j.size + 2) * U32
                A = e @ np.abs(vv) / l
                b_out[t, h] = (A * (2 * rel + 2.0 ** -20) + 2.0 ** -31 * np.abs(vv).sum(0) / l
                               + U16[ftype] * np.abs(out[t, h]) * 1.01 + TINY[ftype])
                b_lse[t, h] = rel + FN + 4 * U32 * (abs(m) + abs(lse[t, h]))
    return out, lse, b_out, b_lse


def head_norm(x, w, eps, w_offset, layer):
    """x [heads][D] -> normed, bound (fp32 sums in a tree over D values)."""
    if w is None:
        return x.copy(), np.zeros_like(x)
    depth = (8 + 5 + 2) * U32       # eight values of a lane, the lanes' tree, the division
    u, eu = x, np.zeros_like(x)
    if layer:
        u = x - x.mean(-1, keepdims=True)
        eu = depth * np.abs(x).mean(-1, keepdims=True) + U32 * np.abs(u)
    ms = (u * u).mean(-1, keepdims=True) + eps
    k = 1 / np.sqrt(ms)
    e_ms = 2 * (np.abs(u) * eu).mean(-1, keepdims=True) + (eu * eu).mean(-1, keepdims=True) + depth * ms
    e_k = k * (e_ms / ms) / 2 * 1.01 + FN * k
    g = np.abs(w + w_offset)
    y = u * k * (w + w_offset)
    return y, g * (k * eu + np.abs(u) * e_k + eu * e_k) + 4 * U32 * np.abs(y) + 2 * U32 * g * np.abs(u) * k


def rotate(x, ex, cos, sin, rot, interleaved):
    y, e = ref.rotate(x, cos, sin, rot, interleaved)
    half = rot // 2
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    c = a + 1 if interleaved else a + half
    ey = ex.copy()
    ey[:, a] = ex[:, a] * np.abs(cos) + ex[:, c] * np.abs(sin)
    ey[:, c] = ex[:, c] * np.abs(cos) + ex[:, a] * np.abs(sin)
    return y, e + ey


def coded(x, ex, factor):
    """What the 4-bit cache holds of x [heads][D], and how far a right store may be off x: half a
    step of the largest right scale, the whole excess where that is clipped, and x's own bound.
    Groups that hold no finite numbers are NaN."""
    g, eg = x.reshape(x.shape[0], -1, 16), ex.reshape(x.shape[0], -1, 16)
    top = np.abs(g).max(-1, keepdims=True) / factor
    with np.errstate(invalid="ignore"):
        big = top * (1 + 1e-5) + (np.abs(eg).max(-1, keepdims=True) / factor)
        want = np.minimum(big / 7, 448.0)
        table = E4M3[:127]
        step = table[np.minimum(np.searchsorted(table, np.nan_to_num(want)), 126)] * factor   # not below the right one
        # a scale rounds down by 2^-4 at most (by half of 2^-9 below 2^-6): the largest code is 7
        clip = np.maximum(np.abs(g) - 7.5 * np.minimum(want * (1 - 2.0 ** -4) - 2.0 ** -10, 448.0).clip(0) * factor, 0)
    bound = step / 2 + clip + eg + 1e-6 * np.abs(g)
    odd = ~np.isfinite(g).all(-1, keepdims=True)
    y = np.where(odd, np.nan, g)
    return y.reshape(x.shape), np.broadcast_to(bound, g.shape).reshape(x.shape)


def head_append(q, k, w_q, w_k, eps, w_offset, layer, positions, cos, sin, interleaved):
    """Normed and rotated q and k [T][heads][D] (zeros where a token is not live), their
    bounds before any rounding into 16 or 4 bits, and which tokens are live."""
    T = k.shape[0]
    rot = 0 if cos is None else 2 * cos.shape[1]
    live = np.array([p >= 0 and (not rot or p < cos.shape[0]) for p in positions])
    outs = []
    for x, w in ((q, w_q), (k, w_k)):
        y, e = np.zeros_like(x), np.zeros_like(x)
        for t in range(T):
            if not live[t]:
                continue
            with np.errstate(invalid="ignore"):
                y[t], e[t] = head_norm(x[t], w, eps, w_offset, layer)
                if rot:
                    y[t], e[t] = rotate(y[t], e[t], cos[positions[t]], sin[positions[t]], rot, interleaved)
        outs += [y, e]
    return outs[0], outs[1], outs[2], outs[3], live


def pages(lens, new, table, pool, state, page, max_tokens):
    """dg_assign_pages, one sequence after the other.  Returns lens, table, pool, state,
    starts, slots, positions."""
    table, pool = table.copy(), pool.copy()
    B, width, N = len(lens), table.shape[1], len(pool)
    out = np.array(lens, np.int64)
    first, count = int(state[0]), int(state[1])
    slots, positions = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int64)
    starts, asked, taken, back = [0], 0, 0, []
    for b in range(B):
        n, w = max(int(lens[b]), 0), int(new[b])
        held = -(-n // page)
        starts.append(starts[-1] + max(w, 0))
        if w < 0:
            back += list(table[b, :min(held, width)])
            out[b] = 0
            continue
        need = -(-(n + w) // page)
        if need > width or (max_tokens and starts[-1] > max_tokens):
            continue
        asked += need - held
        if need > held:
            if asked > count:
                continue
            table[b, held:need] = [pool[(first + taken + i) % N] for i in range(need - held)]
            taken = asked
        out[b] = n + w
        if max_tokens:
            for i in range(w):
                p = n + i
                pg = int(table[b, p // page])
                slots[starts[-2] + i] = -1 if pg < 0 else pg * page + p % page
                positions[starts[-2] + i] = p
    back = back[:N - count]
    for i, pg in enumerate(back):
        pool[(first + count + i) % N] = pg
    return (out, table, pool, np.array([(first + taken) % N, count - taken + len(back)]), np.array(starts), slots,
            positions)


def logprobs(x, tokens, top_k, scale):
    """x float64 [R][V] of the logits' values.  Returns per row lse, logprob, entropy, rank, top_ids,
    top_logprobs and bounds of lse, logprob and entropy (top_logprobs': as logprob's)."""
    R, V = x.shape
    lse, lp, H = (np.zeros(R) for _ in range(3))
    b_lse, b_lp, b_H = (np.zeros(R) for _ in range(3))
    rank, ids, tops = np.zeros(R, np.int64), np.zeros((R, top_k), np.int64), np.zeros((R, top_k))
    for r in range(R):
        z, t = scale * x[r], int(tokens[r])
        number = ~np.isnan(x[r])
        order = np.lexsort((np.arange(V), np.where(number, -np.nan_to_num(x[r], posinf=np.inf, neginf=-np.inf), 0.0),
                            ~number))
        rank[r] = np.flatnonzero(order == t)[0] if 0 <= t < V else V
        ids[r] = order[:top_k]
        if not number.all() or (x[r] == np.inf).any():
            lse[r] = lp[r] = H[r] = np.nan
            tops[r] = np.nan
            continue
        m = z.max()
        if m == -np.inf:
            lse[r], lp[r], tops[r] = -np.inf, -np.inf, -np.inf
            continue
        e = np.exp(z - m)
        l = e.sum()
        with np.errstate(invalid="ignore"):
            d = np.where(e > 0, z - m, 0.0)
        lse[r] = m + np.log(l)
        H[r] = np.log(l) - (e * d).sum() / l
        lp[r] = (z[t] - m) - np.log(l) if 0 <= t < V else -np.inf     # (z - lse cancels for masks of -1e38)
        tops[r] = (z[ids[r]] - m) - np.log(l)
        # an exponent errs by a rounding of its difference, of its product and of the factor; sums run at most
        # 2 * vectors of a thread + 14 roundings deep; scale * (x - m) and the logarithm a few more
        deep = (V / 256 + 64) * U32
        ez = 4 * U32 * (e * np.abs(d)).sum() / l
        b_l = ez + FN + deep
        b_lse[r] = b_l + 4 * U32 * (abs(m) + abs(lse[r]) + 16)
        b_lp[r] = b_l + 4 * U32 * ((abs(lp[r]) if np.isfinite(lp[r]) else 0.0) + 32)
        A = (e * np.abs(d)).sum() / l
        B2 = (e * d * d).sum() / l
        b_H[r] = b_l + A * (2 * FN + 2 * deep + ez) + 4 * U32 * B2 + 8 * U32 * (np.log(l) + A + 16)
    return lse, lp, H, rank, ids, tops, b_lse, b_lp, b_H
