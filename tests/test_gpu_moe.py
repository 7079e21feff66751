"""The mixture-of-experts layer (dg_moe_forward) against the definition in 64
bits: all weight formats, 1..16 tokens, routings that spread, collide and tie,
odd sizes, both scorings, residuals, determinism, streams and graphs."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
KIND = {"f16": dg.LINEAR_F16, "bf16": dg.LINEAR_BF16, "w4": dg.LINEAR_W4A16}


def _case(fmt, M, K, I, E, seed, group=32):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if fmt == "bf16" else torch.float16
    n = lambda shape, std: (torch.randn(shape, generator=g) * std).to(dt)
    t = {"x": n((M, K), 1.0), "router": n((E, K), K ** -0.5), "res": n((M, K), 1.0)}
    for name, r, c in (("gate", I, K), ("up", I, K), ("down", K, I)):
        if fmt == "w4":
            q = torch.randint(-8, 8, (E, r, c), generator=g, dtype=torch.int8)
            t["w_" + name] = ((q[..., 0::2] & 15) | ((q[..., 1::2] & 15) << 4)).view(torch.uint8)
            t["s_" + name] = ((0.1 + torch.rand(E, r, c // group, generator=g)) / (2.5 * c ** 0.5)).half()
        else:
            t["w_" + name], t["s_" + name] = n((E, r, c), c ** -0.5), None
    return t


def _op(t, fmt, top_k, group=32, residual=False, dev=None, **kw):
    d = dev if dev is not None else {k: None if v is None else v.to(DEV) for k, v in t.items()}
    M = t["x"].shape[0]
    y = torch.full_like(d["x"], float("nan"))
    ids = torch.full((M, top_k), -9, dtype=torch.int32, device=DEV)
    wts = torch.full((M, top_k), float("nan"), dtype=torch.float32, device=DEV)
    op = dg.moe(KIND[fmt], d["x"], y, d["router"], d["w_gate"], d["w_up"], d["w_down"], top_k,
                gate_scale=d["s_gate"], up_scale=d["s_up"], down_scale=d["s_down"],
                residual=d["res"] if residual else None, ids=ids, weights=wts, group_size=group, **kw)
    ws = torch.full((dg.moe_workspace_bytes(op),), 255, dtype=torch.uint8, device=DEV)
    return op, ws, y, ids, wts, d


def _check(t, fmt, top_k, group=32, residual=False, score=dg.MOE_SOFTMAX, renormalize=True,
           route_scale=1.0, what="moe"):
    op, ws, y, ids, wts, d = _op(t, fmt, top_k, group, residual, score=score, renormalize=renormalize,
                                 route_scale=route_scale)
    dg.moe_forward(op, ws)
    sync()
    x, router = ref.f64(t["x"]), ref.f64(t["router"])
    rid, rw, bw = ref.route(x, router, top_k, score == dg.MOE_SIGMOID, renormalize,
                            float(np.float32(route_scale)), ids.cpu().numpy())
    ref.check(ref.f64(wts), rw, bw, what + " weights")
    if fmt == "w4":
        mat = lambda n: lambda e: ref.int4(t["w_" + n][e].numpy(), ref.f64(t["s_" + n][e]), group)
    else:
        mat = lambda n: lambda e: ref.f64(t["w_" + n][e])
    ry, by = ref.moe(x, rid, rw, bw, mat("gate"), mat("up"), mat("down"),
                     ref.f64(t["res"]) if residual else None, "bf16" if fmt == "bf16" else "f16")
    ref.check(ref.f64(y), ry, by, what + " y")
    return y, ids, wts


@pytest.mark.parametrize("fmt", ["f16", "bf16", "w4"])
@pytest.mark.parametrize("M,K,I,E,top_k", [
    (1, 256, 128, 8, 2),
    (2, 512, 96, 4, 1),
    (3, 128, 160, 33, 8),
    (5, 1024, 64, 16, 3),
    (8, 64, 256, 8, 8),
    (9, 320, 352, 64, 6),
    (16, 256, 192, 8, 2),
    (16, 1056, 32, 5, 5),
    (7, 32, 32, 1, 1),
])
def test_formats_and_shapes(fmt, M, K, I, E, top_k):
    need_gpu()
    _check(_case(fmt, M, K, I, E, 50 + M), fmt, top_k, residual=M % 2 == 0, what="%s M=%d" % (fmt, M))


@pytest.mark.parametrize("fmt,K,I", [("f16", 8, 8), ("bf16", 24, 40), ("f16", 1000, 136), ("bf16", 264, 1016)])
def test_sizes_of_eight(fmt, K, I):
    need_gpu()
    _check(_case(fmt, 4, K, I, 6, 60), fmt, 2, what="K=%d I=%d" % (K, I))


@pytest.mark.parametrize("group,K,I", [(64, 256, 128), (96, 288, 192), (128, 1024, 256)])
def test_int4_groups(group, K, I):
    need_gpu()
    _check(_case("w4", 6, K, I, 8, 61, group), "w4", 2, group=group, what="group %d" % group)


@pytest.mark.parametrize("fmt", ["f16", "w4"])
def test_larger_layers(fmt):
    need_gpu()
    _check(_case(fmt, 1, 2048, 1024, 16, 62), fmt, 8, what="one token")
    _check(_case(fmt, 11, 1536, 448, 16, 63), fmt, 4, what="eleven tokens")


@pytest.mark.parametrize("score", [dg.MOE_SOFTMAX, dg.MOE_SIGMOID])
@pytest.mark.parametrize("renormalize", [False, True])
def test_scorings(score, renormalize):
    need_gpu()
    _check(_case("f16", 4, 128, 64, 300, 64), "f16", 16, score=score, renormalize=renormalize,
           route_scale=2.5, what="scoring")


@pytest.mark.parametrize("fmt", ["f16", "bf16", "w4"])
def test_all_tokens_on_the_same_experts_and_ties(fmt):
    """Equal rows route alike; equal experts tie, the lowest indexes win."""
    need_gpu()
    t = _case(fmt, 16, 256, 96, 12, 65)
    t["x"][:] = t["x"][0]
    _check(t, fmt, 4, what="one routing")
    t["router"][:] = t["router"][5]
    y, ids, wts = _check(t, fmt, 4, what="ties")
    assert (ids.cpu() == torch.arange(4)).all() and torch.allclose(wts.cpu(), torch.full((16, 4), 0.25))
    assert all(torch.equal(y[0], y[i]) for i in range(16))


def test_zero_and_nan_tokens_leave_the_others_alone():
    need_gpu()
    t = _case("f16", 6, 256, 64, 8, 66)
    clean, _, _ = _check(t, "f16", 2)
    t["x"][2] = 0
    t["x"][4, 17] = float("nan")
    op, ws, y, ids, wts, _ = _op(t, "f16", 2, renormalize=True)
    dg.moe_forward(op, ws)
    sync()
    assert (y[2] == 0).all() and torch.isnan(y[4]).all()
    assert ids[4].tolist() == [0, 1]
    for m in (0, 1, 3, 5):
        ref.check(ref.f64(y[m]), ref.f64(clean[m]), 4 * 2.0 ** -11 * np.abs(ref.f64(clean[m])) + 1e-4, "others")


def test_repeatable_on_any_stream_and_in_a_graph():
    need_gpu()
    t = _case("w4", 5, 512, 128, 16, 67)
    op, ws, y, ids, wts, d = _op(t, "w4", 4, renormalize=True)
    dg.moe_forward(op, ws)
    sync()
    base = y.clone()
    s = torch.cuda.Stream()
    for fill in (0, 77, 255):
        ws.fill_(fill)
        y.fill_(1.0)
        s.wait_stream(torch.cuda.current_stream())
        dg.moe_forward(op, ws, stream=s)
        s.synchronize()
        assert torch.equal(y, base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.moe_forward(op, ws)
    x2 = _case("w4", 5, 512, 128, 16, 68)["x"]
    for x in (x2, t["x"]):
        d["x"].copy_(x.to(DEV))
        graph.replay()
        sync()
    assert torch.equal(y, base)


def test_y_may_be_x_and_the_residual():
    need_gpu()
    t = _case("f16", 3, 256, 64, 8, 69)
    t["res"] = t["x"].clone()
    want, _, _ = _check(t, "f16", 2, residual=True)
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    op = dg.moe(dg.LINEAR_F16, d["x"], d["x"], d["router"], d["w_gate"], d["w_up"], d["w_down"], 2,
                residual=d["x"], renormalize=True)
    ws = torch.empty(dg.moe_workspace_bytes(op), dtype=torch.uint8, device=DEV)
    dg.moe_forward(op, ws)
    sync()
    assert torch.equal(d["x"], want)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "w4"])
@pytest.mark.parametrize("M,top_k", [(16, 1), (9, 3), (13, 4), (16, 4)])
def test_crowded_experts_among_many(fmt, M, top_k):
    """All tokens but one on the same experts, more than are taken at a time."""
    need_gpu()
    t = _case(fmt, M, 256, 96, 64, 67)
    keep = t["x"][1].clone()
    t["x"][:] = t["x"][0]
    t["x"][1] = keep
    y, _, _ = _check(t, fmt, top_k, residual=False, what="crowded")
    assert all(torch.equal(y[0], y[i]) for i in range(2, min(M, 8)))


@pytest.mark.parametrize("K,I", [(576, 192), (1088, 320), (96, 704), (544, 1120)])
def test_int4_sizes_between_chunks(K, I):
    need_gpu()
    _check(_case("w4", 3, K, I, 9, 68), "w4", 2, what="K=%d I=%d" % (K, I))
    _check(_case("w4", 12, K, I, 9, 69), "w4", 3, what="K=%d I=%d, twelve" % (K, I))
