"""The expert layer at the ends of its hidden values' range: what the header states of
large, infinite, NaN and small h."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync
from test_gpu_moe import _case, _check

pytestmark = pytest.mark.gpu
KIND = {"f16": dg.LINEAR_F16, "bf16": dg.LINEAR_BF16, "w4": dg.LINEAR_W4A16}


def _pack(q):
    return ((q[..., 0::2] & 15) | ((q[..., 1::2] & 15) << 4)).view(torch.uint8)


def _run(fmt, x, router, gate, up, down, scales=None):
    """One expert a token.  gate, up, down: 16-bit matrices, or (w4) int8 codes with
    one scale a matrix in `scales`."""
    on = lambda t: t.contiguous().to(DEV)
    y = torch.full_like(x, float("nan")).to(DEV)
    kw = {}
    if fmt == "w4":
        full = lambda q, s: on(torch.full(q.shape[:2] + (q.shape[2] // 32,), s, dtype=torch.float16))
        kw = dict(gate_scale=full(gate, scales[0]), up_scale=full(up, scales[1]), down_scale=full(down, scales[2]))
        gate, up, down = _pack(gate), _pack(up), _pack(down)
    held = [on(x), y, on(router), on(gate), on(up), on(down)]
    op = dg.moe(KIND[fmt], *held, 1, **kw, renormalize=True)
    ws = torch.full((dg.moe_workspace_bytes(op),), 255, dtype=torch.uint8, device=DEV)
    dg.moe_forward(op, ws)
    sync()
    return ref.f64(y)


def _large(fmt, tokens, K, I, hot, seed):
    """One expert; token 0's h is hot * hot at index 5, the others' are small."""
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if fmt == "bf16" else torch.float16
    x = (torch.randn(tokens, K, generator=g) * 0.1).to(dt)
    x[:, 0] = 0
    router = torch.zeros(1, K, dtype=dt)
    if fmt == "w4":
        gate, up, down = (torch.randint(-7, 8, (1, r, c), generator=g, dtype=torch.int8)
                          for r, c in ((I, K), (I, K), (K, I)))
        down[down == 0] = 3
        gate[0, :, 0] = up[0, :, 0] = 0
        gate[0, 5, 0] = up[0, 5, 0] = 1
        scales = (2.0, 2.0, 2.0 ** -12)
        x[0, 0] = hot / 2
        real = [q[0].double().numpy() * s for q, s in zip((gate, up, down), scales)]
    else:
        gate, up, down = ((torch.randn(1, r, c, generator=g) * s).to(dt)
                          for r, c, s in ((I, K, 0.1), (I, K, 0.1), (K, I, 2.0 ** -12)))
        down[down == 0] = 2.0 ** -12
        gate[0, :, 0] = up[0, :, 0] = 0
        top = 2.0 ** 60 if fmt == "bf16" else 512.0
        gate[0, 5, 0] = up[0, 5, 0] = top
        x[0, 0] = hot / top
        scales, real = None, [ref.f64(w[0]) for w in (gate, up, down)]
    return (x, router, gate, up, down, scales), real


def _h(x, gate, up):
    g, u = gate @ x, up @ x
    s = g / (1 + np.exp(-g))
    e = lambda W: (x.size + 1) * ref.U32 * (np.abs(W) @ np.abs(x))
    return s * u, 1.1 * e(gate) * np.abs(u) + np.abs(s) * e(up) + 1.1 * e(gate) * e(up) + ref.FN * np.abs(s * u)


@pytest.mark.parametrize("tokens", [1, 2, 4, 12])
@pytest.mark.parametrize("fmt,hot", [("f16", 4120.0), ("f16", 30000.0), ("w4", 4120.0), ("w4", 30000.0),
                                     ("bf16", 2.0 ** 64), ("bf16", 2.0 ** 90)])
def test_hidden_values_past_the_range_become_infinite(fmt, tokens, hot):
    """fp16: 2^24 and more; bf16: what fp32 does not hold.  The output is infinite with
    the down weight's sign; the other tokens of the expert are as without."""
    need_gpu()
    args, real = _large(fmt, tokens, 64, 96, hot, 70)
    y = _run(fmt, *args)
    assert np.array_equal(y[0], np.sign(real[2][:, 5]) * np.inf)
    assert np.isfinite(y[1:]).all()
    args[0][0] = 0
    calm = _run(fmt, *args)
    assert np.array_equal(y[1:], calm[1:])


@pytest.mark.parametrize("tokens", [1, 3, 12])
@pytest.mark.parametrize("fmt", ["f16", "w4"])
def test_hidden_values_just_inside_the_range(fmt, tokens):
    need_gpu()
    args, real = _large(fmt, tokens, 64, 96, 4060.0, 71)     # h about 0.98 * 2^24
    y = _run(fmt, *args)
    h, eh = _h(ref.f64(args[0][0]), real[0], real[1])
    assert 2.0 ** 23.9 < h[5] < 2.0 ** 24
    A = np.abs(real[2]) @ np.abs(h)
    ry = real[2] @ h
    bound = (np.abs(real[2]) @ (eh + 2.0 ** -22 * np.abs(h) + 2.0 ** -28) + 120 * ref.U32 * A
             + ref.U16["f16"] * np.abs(ry) + ref.TINY["f16"])
    ref.check(y[0], ry, bound, "y")


@pytest.mark.parametrize("fmt", ["f16", "bf16", "w4"])
def test_a_nan_hidden_value_is_its_tokens_alone(fmt):
    need_gpu()
    args, _ = _large(fmt, 4, 64, 96, 1.0, 72)
    calm = _run(fmt, *args)
    args[0][2, 9] = float("nan")
    y = _run(fmt, *args)
    assert np.isnan(y[2]).all()
    assert np.array_equal(y[[0, 1, 3]], calm[[0, 1, 3]])


@pytest.mark.parametrize("tokens", [1, 2, 4, 12])
@pytest.mark.parametrize("fmt", ["f16", "w4"])
@pytest.mark.parametrize("size", [2.0 ** -6, 2.0 ** -10, 2.0 ** -14, 2.0 ** -18])
def test_small_hidden_values_keep_the_stated_steps(fmt, tokens, size):
    """Gate and up of `size` and large down weights: h is held to 22 bits, or to steps
    of 2^-27."""
    need_gpu()
    K, I = 128, 160
    g = torch.Generator().manual_seed(73)
    x = torch.randn(tokens, K, generator=g).half()
    if fmt == "w4":
        gate, up, down = (torch.randint(-7, 8, (1, r, c), generator=g, dtype=torch.int8)
                          for r, c in ((I, K), (I, K), (K, I)))
        scales = tuple(float(np.float16(s)) for s in (0.25, size * K ** -0.5 / 4, 16.0))
        real = [q[0].double().numpy() * s for q, s in zip((gate, up, down), scales)]
    else:
        gate, up, down = ((torch.randn(1, r, c, generator=g) * s).half()
                          for r, c, s in ((I, K, 1.0), (I, K, size * K ** -0.5), (K, I, 64.0)))
        scales, real = None, [ref.f64(w[0]) for w in (gate, up, down)]
    y = _run(fmt, x, torch.zeros(1, K).half(), gate, up, down, scales)
    for m in range(tokens):
        h, eh = _h(ref.f64(x[m]), real[0], real[1])
        A = np.abs(real[2]) @ np.abs(h)
        ry = real[2] @ h
        bound = (np.abs(real[2]) @ (eh + 2.0 ** -22 * np.abs(h) + 2.0 ** -28) + (I + 20) * ref.U32 * A
                 + ref.U16["f16"] * np.abs(ry) + ref.TINY["f16"])
        ref.check(y[m], ry, bound, "token %d" % m)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "w4"])
@pytest.mark.parametrize("M,top_k,E", [(8, 1, 8), (8, 3, 5), (16, 4, 7), (2, 2, 16)])
def test_a_token_changes_its_place_from_expert_to_expert(fmt, M, top_k, E):
    """Each expert's list of tokens differs, so that the sums of one token come from
    other lanes of a warp expert by expert; short rows, so that a warp has the chunks
    of many experts.  The same bits on every call."""
    need_gpu()
    t = _case(fmt, M, 512, 32, E, 74)
    first, ids, _ = _check(t, fmt, top_k, residual=True, what="first")
    lists = [np.argwhere((ids.cpu().numpy() == e).any(1))[:, 0].tolist() for e in range(E)]
    places = {m: {held.index(m) for held in lists if m in held} for m in range(M)}
    assert top_k == 1 or M == 2 or any(len(p) > 1 for p in places.values())
    for _ in range(3):
        again, _, _ = _check(t, fmt, top_k, residual=True, what="again")
        assert torch.equal(again, first)
