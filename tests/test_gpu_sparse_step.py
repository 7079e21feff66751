"""A sparse decoder's step: every stage against the definition in 64 bits from
the values that the device held, several tokens a step and single ones, int4
experts, windows, several sequences, and the captured graph."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync
from quantized_skinny_gemm_gb300 import plans, synth

pytestmark = pytest.mark.gpu
HEADS, KV_HEADS, DIM, HIDDEN, INTER, EXPERTS, TOP_K = 6, 2, 64, 256, 96, 8, 3
EPS = float(np.float32(1e-6))


def _layers(int4=False, layers=2):
    return synth.sparse_decoder_workload(3, layers, HIDDEN, HEADS, KV_HEADS, DIM, INTER, EXPERTS, int4)


def _product(W, x, got, what):
    W, x = ref.f64(W), ref.f64(x)
    y = x @ W.T
    ref.check(ref.f64(got), y, W.shape[1] * ref.U32 * (np.abs(x) @ np.abs(W).T) + ref.U16["f16"] * np.abs(y)
              + ref.TINY["f16"], what)


def _check_step(step, layers, before, q_len, rope, window=0, sinks=0):
    """before: the caches as they were, in 64 bits."""
    h, y = step.h, None
    table, lens = step.block_table.cpu().numpy(), step.seq_lens.cpu().numpy()
    cos, sin = ref.f64(rope[0]), ref.f64(rope[1])
    T = step.h.shape[0]

    def norm(h, y, w, h_out, x_out, what):
        rh, rx, bh, bx = ref.norm(ref.f64(h), None if y is None else ref.f64(y), ref.f64(w), None, None, None, None,
                                  1.0, 1.0, EPS, 0.0, False, "f16", True)
        ref.check(ref.f64(h_out), rh, bh, what + " h")
        ref.check(ref.f64(x_out), rx, bx, what + " x")

    for i, (L, t, (kd, vd), (kb, vb)) in enumerate(zip(layers, step.layers, step.caches, before)):
        what = "layer %d " % i
        norm(h, y, L.norm_attn, t["h"], t["x"], what + "norm before attention")
        for n in "qkv":
            _product(getattr(L, n), t["x"], t[n], what + n)
        rows = lambda n, heads: ref.f64(t[n]).reshape(T, heads, DIM)
        rq, rk, rv, bq, bk = ref.append(rows("q", HEADS), rows("k", KV_HEADS), rows("v", KV_HEADS), kb, vb, table, lens,
                                        q_len, cos, sin, False, "f16")
        ref.check(rows("q_rot", HEADS), rq, bq, what + "rotated q")
        ref.check(ref.f64(kd), rk, bk, what + "keys")
        assert np.array_equal(ref.f64(vd), rv)
        ro, _, bo, _ = ref.attention(rows("q_rot", HEADS), ref.f64(kd), ref.f64(vd), table, lens, q_len, DIM ** -0.5,
                                     window, sinks)
        ref.check(rows("att", HEADS), ro, bo, what + "attention")
        _product(L.o, t["att"], t["o"], what + "o")
        norm(t["h"], t["o"], L.norm_mlp, t["h_mid"], t["x_mid"], what + "norm before the experts")
        x = ref.f64(t["x_mid"])
        ids, w, bw = ref.route(x, ref.f64(L.router), TOP_K, False, True, 1.0, t["ids"].cpu().numpy())
        ref.check(ref.f64(t["weights"]), w, bw, what + "routing")
        mat = lambda n: lambda e: (ref.int4(getattr(L, n)[e].numpy(), ref.f64(L.scales[n][e]), 32) if L.scales
                                   else ref.f64(getattr(L, n)[e]))
        ry, by = ref.moe(x, ids, w, bw, mat("gate"), mat("up"), mat("down"), None, "f16")
        ref.check(ref.f64(t["y"]), ry, by, what + "experts")
        h, y = t["h_mid"], t["y"]
    norm(h, y, torch.ones(HIDDEN), step.h_out, step.x_out, "last norm")


def _caches(step):
    return [(ref.f64(k), ref.f64(v)) for k, v in step.caches]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("batch,q_len,window,sinks", [(1, 1, 0, 0), (1, 9, 0, 0), (3, 2, 0, 0), (2, 4, 7, 2)])
def test_steps(int4, batch, q_len, window, sinks):
    """Three steps on, with ragged lengths and pages in no order."""
    need_gpu()
    layers, rope = _layers(int4), synth.rotary_tables(128, DIM)
    step = plans.sparse_decoder_step(layers, DEV, HEADS, KV_HEADS, TOP_K, batch=batch, q_len=q_len, page_size=16,
                                     max_pages=4, window=window, sinks=sinks, rope=rope)
    g = torch.Generator().manual_seed(9)
    step.block_table.copy_(torch.randperm(batch * 4, generator=g).view(batch, 4).int())
    step.seq_lens.copy_(torch.arange(batch).int() * 5)
    for _ in range(3):
        before = _caches(step)
        step.seq_lens += q_len
        step.h.copy_(torch.randn(batch * q_len, HIDDEN, generator=g))
        step.run()
        sync()
        _check_step(step, layers, before, q_len, rope, window, sinks)


def test_a_window_of_tokens_and_single_ones_share_the_caches():
    need_gpu()
    layers, rope = _layers(), synth.rotary_tables(64, DIM)
    one = plans.sparse_decoder_step(layers, DEV, HEADS, KV_HEADS, TOP_K, page_size=16, max_pages=4, rope=rope)
    many = plans.sparse_decoder_step(layers, DEV, HEADS, KV_HEADS, TOP_K, q_len=11, page_size=16, max_pages=4,
                                     rope=rope, share=one)
    g = torch.Generator().manual_seed(10)
    for step, n in ((many, 11), (one, 1), (many, 11), (one, 1)):
        before = _caches(one)
        one.seq_lens += n
        step.h.copy_(torch.randn(n, HIDDEN, generator=g))
        step.run()
        sync()
        _check_step(step, layers, before, n, rope)
    assert one.seq_lens.tolist() == [24]
    with pytest.raises(ValueError):
        plans.sparse_decoder_step(layers, DEV, HEADS, KV_HEADS, TOP_K, batch=2, share=one)


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("prompt", [1, 16, 37])
def test_the_example_decodes_the_same_in_a_graph(int4, prompt):
    need_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import sparse_decode
    layers = _layers(int4, 3)
    g = torch.Generator().manual_seed(11)
    embed, lm_head = synth.normal((512, HIDDEN), 1.0, g), synth.normal((512, HIDDEN), HIDDEN ** -0.5, g)
    words = torch.randint(0, 512, (prompt,), generator=g)
    runs = [sparse_decode.decode(layers, embed, lm_head, words, 20, HEADS, KV_HEADS, TOP_K, DEV, graph)[0]
            for graph in (True, False, True)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])
    assert (runs[0] >= 0).all() and (runs[0] < 512).all()
