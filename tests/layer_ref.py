"""The decoder-layer operators' definitions in 64 bits, with error bounds.

TEST INFRASTRUCTURE ONLY.  Everything is numpy float64 on the host, one row at
a time, from the definitions in include/dg.h.  Each function also returns the
bound its 16- or 32-bit outputs are held to, derived from the arithmetic that
the header promises (fp32 sums, one rounding into the output):

  u16      unit roundoff of the 16-bit type: 2^-11 (fp16), 2^-8 (bf16)
  sums     n terms in fp32: n * 2^-24 * sum |term|
  functions (exp, division, square root, silu): 2^-20 relative, as for the
            library's epilogues
"""
import numpy as np

U16 = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -133}   # smallest step of the output type
U32 = 2.0 ** -24
FN = 2.0 ** -20


def f64(t):
    return t.detach().cpu().double().numpy()


def visible(p, capacity, pages, page_size, window, sinks):
    j = np.arange(max(0, min(p + 1, capacity)))
    keep = pages[j // page_size] >= 0
    if window:
        keep &= (j > p - window) | (j < sinks)
    return j[keep]


def attention(q, k_cache, v_cache, table, lens, q_len, scale, window=0, sinks=0, ftype="f16"):
    """q [T][H][D] float64, caches [P][S][G][D] float64, table int [B][max],
    lens int [B] -> out, lse, bound of out, bound of lse."""
    T, H, D = q.shape
    P, S, G, _ = k_cache.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    b_out, b_lse = np.full((T, H, D), TINY[ftype]), np.zeros((T, H))
    table = np.where((table >= 0) & (table < P), table, -1)
    for t in range(T):
        b = t // q_len
        p = int(lens[b]) - q_len + t % q_len
        j = visible(p, table.shape[1] * S, table[b], S, window, sinks)
        if not j.size:
            continue
        pg, sl = table[b][j // S], j % S
        for h in range(H):
            k, v = k_cache[pg, sl, h // (H // G)], v_cache[pg, sl, h // (H // G)]
            with np.errstate(invalid="ignore", over="ignore"):
                z = scale * (k @ q[t, h])
                m = z.max()
                if m == -np.inf:
                    continue
                e = np.exp(z - m)
                l = e.sum()
                out[t, h] = e @ v / l
                lse[t, h] = m + np.log(l)
                # a score errs by D fp32 roundings of its products and one of the
                # scale; each weight by that, by its function and by its 16-bit
                # rounding (absolute 2^-25 where it is fp16-subnormal)
                ez = (D + 2) * U32 * abs(scale) * (np.abs(k) @ np.abs(q[t, h])) + U32 * np.abs(z)
                rel = ez.max() + FN + (j.size + 2) * U32
                A = e @ np.abs(v) / l
                b_out[t, h] = (A * (2 * rel + 2 * U16[ftype]) + 2.0 ** -24 * np.abs(v).sum(0) / l
                               + U16[ftype] * np.abs(out[t, h]) + TINY[ftype])
                b_lse[t, h] = rel + FN + 2 * U32 * (abs(m) + abs(lse[t, h]))
    return out, lse, b_out, b_lse


def rotate(x, cos, sin, rot, interleaved):
    """x [heads][D] float64 -> rotated, bound of the fp32 evaluation."""
    y, e = x.copy(), np.zeros_like(x)
    half = rot // 2
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    c = a + 1 if interleaved else a + half
    y[:, a] = x[:, a] * cos - x[:, c] * sin
    y[:, c] = x[:, c] * cos + x[:, a] * sin
    e[:, a] = 2 * U32 * (np.abs(x[:, a] * cos) + np.abs(x[:, c] * sin))
    e[:, c] = 2 * U32 * (np.abs(x[:, c] * cos) + np.abs(x[:, a] * sin))
    return y, e


def append(q, k, v, k_cache, v_cache, table, lens, q_len, cos, sin, interleaved, ftype):
    """Returns q_out, k_cache, v_cache (float64 copies, updated), bounds of
    q_out and k_cache (v and untouched slots are exact)."""
    T = k.shape[0]
    P, S = k_cache.shape[:2]
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    b_k = np.zeros_like(k_cache)
    q_out = np.zeros_like(q)
    b_q = np.zeros_like(q)
    rot = 0 if cos is None else 2 * cos.shape[1]
    for t in range(T):
        p = int(lens[t // q_len]) - q_len + t % q_len
        if p < 0 or (rot and p >= cos.shape[0]):
            continue
        c, s = (cos[p], sin[p]) if rot else (np.zeros(0), np.zeros(0))
        yq, eq = rotate(q[t], c, s, rot, interleaved)
        yk, ek = rotate(k[t], c, s, rot, interleaved)
        q_out[t] = yq
        b_q[t] = eq + U16[ftype] * np.abs(yq) + TINY[ftype]
        if p // S >= table.shape[1]:
            continue
        page = table[t // q_len][p // S]
        if not 0 <= page < P:
            continue
        k_cache[page, p % S] = yk
        v_cache[page, p % S] = v[t]
        b_k[page, p % S] = ek + U16[ftype] * np.abs(yk) + TINY[ftype]
    return q_out, k_cache, v_cache, b_q, b_k


def _norm(v, ev, w, b, eps, w_offset, layer):
    """norm(v; w, b) and its bound, where v errs by ev.  Sums over a row run in
    at most 32 + 32 + 10 roundings deep (registers, then a tree)."""
    depth = 74 * U32
    N = v.shape[-1]
    u, eu = v, ev
    if layer:
        u = v - v.mean(-1, keepdims=True)
        eu = ev + ev.mean(-1, keepdims=True) + depth * np.abs(v).mean(-1, keepdims=True) + U32 * np.abs(u)
    ms = (u * u).mean(-1, keepdims=True) + eps
    k = 1 / np.sqrt(ms)
    e_ms = 2 * (np.abs(u) * eu).mean(-1, keepdims=True) + (eu * eu).mean(-1, keepdims=True) + depth * ms
    e_k = k * (e_ms / ms) / 2 * 1.01 + FN * k
    g = np.abs(w + w_offset)
    x = u * k * (w + w_offset) + (b if b is not None else 0.0)
    ex = g * (k * eu + np.abs(u) * e_k + eu * e_k) + 6 * U32 * (g * np.abs(u) * k + np.abs(x))
    return x, ex


def norm(h, y, w_pre, b_pre, w_post, b_post, gate, alpha, beta, eps, w_offset, layer, ftype, h_f32):
    """Returns h', x and their bounds (x is None without w_pre)."""
    v, ev = 0.0, 0.0
    if y is not None:
        r, er = y, np.zeros_like(y)
        if w_post is not None:
            r, er = _norm(r, er, w_post, b_post, eps, w_offset, layer)
        if gate is not None:
            r, er = r * gate, er * np.abs(gate) + U32 * np.abs(r * gate)
        v, ev = beta * r, abs(beta) * er + 2 * U32 * np.abs(beta * r)
    if h is not None:
        v, ev = v + alpha * h, ev + U32 * np.abs(alpha * h)
    ev = ev + U32 * np.abs(v)
    u_h = U32 if h_f32 else U16[ftype]
    b_h = ev + u_h * np.abs(v) + (0.0 if h_f32 else TINY[ftype])
    if w_pre is None:
        return v, None, b_h, None
    x, ex = _norm(v, ev, w_pre, b_pre, eps, w_offset, layer)
    return v, x, b_h, ex + U16[ftype] * np.abs(x) + TINY[ftype]


def int4(packed, scales, group):
    """packed uint8 [..., cols / 2], scales [..., cols / group] -> float64."""
    lo, hi = (packed & 15).astype(np.int64), (packed >> 4).astype(np.int64)
    q = np.stack((lo, hi), -1).reshape(packed.shape[:-1] + (-1,))
    q = np.where(q > 7, q - 16, q).astype(np.float64)
    return q * np.repeat(scales, group, axis=-1)


def route(x, router, top_k, sigmoid, renormalize, route_scale, got=None):
    """ids, weights (float64) and the weights' bound.  Where a token's scores
    lie nearer than their fp32 bound, its choice is open: `got`'s is taken if
    every expert in it could stand there."""
    z = x @ router.T
    ez = (x.shape[1] + 1) * U32 * (np.abs(x) @ np.abs(router).T).max(1, keepdims=True)
    if sigmoid:
        p = 1 / (1 + np.exp(-z))
    else:
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    ids = np.argsort(-p, axis=1, kind="stable")[:, :top_k]
    if got is not None:
        for m in np.argwhere((got != ids).any(1))[:, 0]:
            assert len(set(got[m])) == top_k and (0 <= got[m]).all() and (got[m] < z.shape[1]).all()
            assert (z[m, got[m]] != z[m, ids[m]]).sum() == (got[m] != ids[m]).sum(), "a tie went up"
            assert (np.abs(z[m, got[m]] - z[m, ids[m]]) <= 2 * ez[m]).all(), "token %d's experts" % m
            ids[m] = got[m]
    w = np.take_along_axis(p, ids, 1)
    b_w = 4 * ez + 4 * FN
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    return ids, w * route_scale, b_w * np.abs(w * route_scale)


def moe(x, ids, weights, b_w, gate, up, down, residual, ftype):
    """gate, up, down: functions e -> float64 matrix.  Returns y and its bound."""
    M, K = x.shape
    y = np.zeros((M, K)) if residual is None else residual.copy()
    err = U32 * np.abs(y)
    u_h = {"f16": 2.0 ** -21, "bf16": 2.0 ** -15}[ftype]   # h as two 16-bit values
    for m in range(M):
        for c, e in enumerate(ids[m]):
            Wg, Wu, Wd = gate(e), up(e), down(e)
            I = Wg.shape[0]
            g, u = Wg @ x[m], Wu @ x[m]
            eg = (K + 1) * U32 * (np.abs(Wg) @ np.abs(x[m]))
            eu = (K + 1) * U32 * (np.abs(Wu) @ np.abs(x[m]))
            s = g / (1 + np.exp(-g))
            h = s * u
            eh = 1.1 * eg * np.abs(u) + np.abs(s) * eu + 1.1 * eg * eu + (FN + u_h) * np.abs(h) + 2.0 ** -26
            A = np.abs(Wd) @ np.abs(h)
            part = Wd @ h
            y[m] += weights[m, c] * part
            err[m] += (abs(weights[m, c]) * (np.abs(Wd) @ eh + (I + 20) * U32 * A)
                       + b_w[m, c] * np.abs(part))
    return y, err + U16[ftype] * np.abs(y) + TINY[ftype]


def check(got, ref, bound, what):
    """NaN and infinities where the reference has them, else within the bound."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what + ": NaN in other places"
    odd = ~fine & ~np.isnan(ref)
    assert np.array_equal(got[odd], ref[odd]), what + ": infinities differ"
    err = np.abs(np.where(fine, got, 0.0) - np.where(fine, ref, 0.0))
    bad = fine & ~(err <= np.broadcast_to(bound, ref.shape))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d outside; first at %s: %r, ref %r, bound %r" % (
            what, bad.sum(), bad.size, i, got[i], ref[i], np.broadcast_to(bound, ref.shape)[i]))
