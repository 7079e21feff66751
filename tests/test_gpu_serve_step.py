"""A sparse decoder's step with norms of the heads, a 4-bit cache and pages from a pool: every
stage against the definitions in 64 bits from the values that the device held, sequences that grow
into new pages, end and are refused, the captured graph, and the example."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
import serve_ref
from gpu_util import DEV, need_gpu, sync
from quantized_skinny_gemm_gb300 import plans, synth

pytestmark = pytest.mark.gpu
HEADS, KV_HEADS, DIM, HIDDEN, INTER, EXPERTS, TOP_K, PAGE = 6, 2, 64, 256, 96, 8, 3, 16
EPS = float(np.float32(1e-6))
KF, VF = 0.5, 0.25


def _layers(layers=2, head_norms=True):
    return synth.sparse_decoder_workload(3, layers, HIDDEN, HEADS, KV_HEADS, DIM, INTER, EXPERTS, head_norms=head_norms)


def _step(bits, batch, q_len, pool_pages, rope, layers=None, **kw):
    return plans.sparse_decoder_step(layers or _layers(), DEV, HEADS, KV_HEADS, TOP_K, batch=batch, q_len=q_len,
                                     page_size=PAGE, max_pages=4, rope=rope, cache_bits=bits, k_factor=KF, v_factor=VF,
                                     pool_pages=pool_pages, **kw)


def _state(step):
    n = lambda t: t.cpu().numpy().copy()
    return n(step.seq_lens), n(step.block_table), n(step.pool), n(step.pool_state)


def _held(cache):
    """A layer's cache as it is on the device, in 64 bits."""
    if len(cache) == 2:
        return [ref.f64(t) for t in cache]
    k, v, ks, vs = (t.cpu().numpy() for t in cache)
    return serve_ref.decode4(k, ks, KF), serve_ref.decode4(v, vs, VF)


def _check_step(step, before, caches, bits, q_len, rope, layers):
    """before: lengths, table, pool and state; caches: what the caches held."""
    batch = step.seq_lens.numel()
    T = batch * q_len
    want = serve_ref.pages(before[0], np.full(batch, q_len), before[1], before[2], before[3], PAGE, T)
    for name, got, w in zip(("lens", "table", "pool", "state"), _state(step), want):
        assert np.array_equal(got, w), name
    slots, pos = want[5], want[6]
    assert np.array_equal(step.slots.cpu().numpy(), slots) and np.array_equal(step.positions.cpu().numpy(), pos)
    cos, sin = ref.f64(rope[0]), ref.f64(rope[1])
    lens, table = want[0], want[1]
    served = np.repeat(lens > before[0], q_len)
    written = slots >= 0
    for L, t, cache, was in zip(layers, step.layers, step.caches, caches):
        rows = lambda n, heads: ref.f64(t[n]).reshape(T, heads, DIM)
        q, eq, k, ek, live = serve_ref.head_append(rows("q", HEADS), rows("k", KV_HEADS), ref.f64(L.norm_q),
                                                   ref.f64(L.norm_k), EPS, 0.0, False, pos, cos, sin, False)
        ref.check(rows("q_rot", HEADS), q, eq + ref.U16["f16"] * (np.abs(q) + eq) + ref.TINY["f16"], "q")
        now = _held(cache)
        v = rows("v", KV_HEADS)
        for name, held, old, x, ex, f in (("k", now[0], was[0], k, ek, KF), ("v", now[1], was[1], v, 0 * v, VF)):
            flat, flat_was = (c.reshape(-1, KV_HEADS, DIM) for c in (held, old))
            rest = np.setdiff1d(np.arange(len(flat)), slots[written])
            assert np.array_equal(flat[rest], flat_was[rest]), name + ": a place that no token owns"
            if not written.any():
                continue
            if bits == 4:
                w = [serve_ref.coded(x[i], ex[i], f) for i in np.flatnonzero(written)]
                ref.check(flat[slots[written]], np.stack([a for a, _ in w]), np.stack([b for _, b in w]), name)
            else:
                ref.check(flat[slots[written]], x[written],
                          (ex + ref.U16["f16"] * (np.abs(x) + ex) + ref.TINY["f16"])[written], name)
        args = (rows("q_rot", HEADS), now[0], now[1], table, lens, q_len, DIM ** -0.5)
        ro, _, bo, _ = serve_ref.attention4(*args) if bits == 4 else ref.attention(*args)
        ref.check(rows("att", HEADS)[served], ro[served], bo[served], "attention")


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("batch,q_len,pool_pages", [(1, 1, 4), (3, 2, 9), (2, 5, 5), (4, 4, 6)])
def test_steps_from_a_pool(bits, batch, q_len, pool_pages):
    """Sequences grow until the pool or their tables are full; one ends on the way and its
    pages go to others."""
    need_gpu()
    layers, rope = _layers(), synth.rotary_tables(64, DIM)
    step = _step(bits, batch, q_len, pool_pages, rope, layers)
    assert (step.block_table == -1).all() and step.pool_state.tolist() == [0, pool_pages]
    g = torch.Generator().manual_seed(9)
    refused = 0
    for turn in range(64 // q_len + 3):
        step.h.copy_(torch.randn(batch * q_len, HIDDEN, generator=g))
        before, caches = _state(step), [_held(c) for c in step.caches]
        step.run()
        sync()
        if turn % 3 == 0 or turn > 40 // q_len:
            _check_step(step, before, caches, bits, q_len, rope, layers)
        refused += int((step.positions < 0).any())
        if turn == 20 // q_len and batch > 1:
            before = _state(step)
            gone = np.zeros(batch, np.int64)
            gone[1] = -1
            step.end(torch.from_numpy(gone).int().to(DEV))
            sync()
            want = serve_ref.pages(before[0], gone, before[1], before[2], before[3], PAGE, 0)
            for got, w in zip(_state(step), want):
                assert np.array_equal(got, w)
            assert step.seq_lens[1].item() == 0
    lens, table, pool, state = _state(step)
    assert refused
    used = [p for b in range(batch) for p in table[b, :-(-lens[b] // PAGE)]]
    assert sorted(used + [pool[(state[0] + i) % pool_pages] for i in range(state[1])]) == list(range(pool_pages))


def test_a_window_and_single_tokens_share_pool_and_cache():
    need_gpu()
    layers, rope = _layers(), synth.rotary_tables(64, DIM)
    one = _step(4, 1, 1, 4, rope, layers)
    many = plans.sparse_decoder_step(layers, DEV, HEADS, KV_HEADS, TOP_K, q_len=11, rope=rope, share=one, max_pages=4,
                                     cache_bits=4, k_factor=KF, v_factor=VF)
    g = torch.Generator().manual_seed(10)
    for step, n in ((many, 11), (one, 1), (many, 11), (one, 1)):
        step.h.copy_(torch.randn(n, HIDDEN, generator=g))
        before, caches = _state(one), [_held(c) for c in one.caches]
        step.run()
        sync()
        _check_step(step, before, caches, 4, n, rope, layers)
    assert one.seq_lens.tolist() == [24]


def test_a_graph_of_the_step_and_its_log_probabilities():
    """One captured graph of a whole step and what is said of its token, replayed while sequences
    grow, against the same calls one by one."""
    need_gpu()
    layers, rope = _layers(), synth.rotary_tables(64, DIM)
    V = 1000
    head = synth.normal((V, HIDDEN), HIDDEN ** -0.5, torch.Generator().manual_seed(1)).to(DEV)
    runs = []
    for graph in (False, True):
        step = _step(4, 1, 1, 4, rope, layers)
        logits, token = torch.empty(V, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
        lp = {"logprob": torch.empty(1, device=DEV), "rank": torch.empty(1, dtype=torch.int32, device=DEV),
              "entropy": torch.empty(1, device=DEV), "top_ids": torch.empty(1, 4, dtype=torch.int32, device=DEV),
              "top_logprobs": torch.empty(1, 4, device=DEV)}
        op = dg.linear(dg.LINEAR_F16, head, 1, V, HIDDEN, x=step.x_out, logits=logits, token=token)
        ws = torch.empty(dg.workspace_bytes([op]), dtype=torch.uint8, device=DEV)
        say = dg.logprobs(logits, tokens=token, **lp)
        ws2 = torch.empty(max(16, dg.logprobs_workspace_bytes(say)), dtype=torch.uint8, device=DEV)

        def turn():
            step.run()
            dg.lm_head_argmax(op, ws)
            dg.token_logprobs(say, ws2)
        call = turn
        if graph:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                turn()
            call = captured.replay
        g, seen = torch.Generator().manual_seed(11), []
        for _ in range(40):
            step.h.copy_(torch.randn(1, HIDDEN, generator=g))
            call()
            sync()
            seen.append([logits.clone(), token.clone()] + [t.clone() for t in lp.values()] + [step.seq_lens.clone()])
            want = torch.log_softmax(logits.double(), 0)
            assert lp["rank"].item() == 0 and lp["top_ids"][0, 0] == token
            assert abs(lp["logprob"].item() - want[token.long()].item()) < 1e-4
            assert abs(lp["entropy"].item() + (want.exp() * want).sum().item()) < 1e-4
        runs.append(seen)
    for a, b in zip(*runs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals():
    need_gpu()
    layers, rope = _layers(), synth.rotary_tables(64, DIM)
    one = _step(4, 1, 1, 4, rope, layers)
    for kw in (dict(cache_bits=8), dict(cache_bits=16, share=one), dict(cache_bits=4, share=one, pool_pages=3),
               dict(pool_pages=0)):
        with pytest.raises(ValueError):
            plans.sparse_decoder_step(layers, DEV, HEADS, KV_HEADS, TOP_K, rope=rope, **kw)


@pytest.mark.parametrize("prompt", [1, 37])
@pytest.mark.parametrize("bits,pool,head_norms,logprobs", [(4, True, True, 5), (4, False, False, 0), (16, True, True, 32),
                                                          (16, False, True, 1)])
def test_the_example_decodes_the_same_in_a_graph(prompt, bits, pool, head_norms, logprobs):
    need_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import sparse_decode
    layers = _layers(3, head_norms)
    g = torch.Generator().manual_seed(11)
    embed, lm_head = synth.normal((512, HIDDEN), 1.0, g), synth.normal((512, HIDDEN), HIDDEN ** -0.5, g)
    words = torch.randint(0, 512, (prompt,), generator=g)
    runs = [sparse_decode.decode(layers, embed, lm_head, words, 40, HEADS, KV_HEADS, TOP_K, DEV, graph, bits, pool, logprobs)
            for graph in (True, False)]
    assert torch.equal(runs[0][0], runs[1][0])
    if logprobs:
        a, b = runs[0][2], runs[1][2]
        assert all(torch.equal(a[k], b[k]) for k in a)
        assert (a["rank"] == 0).all() and torch.equal(a["top_ids"][:, 0], runs[0][0])
        assert torch.equal(a["top_logprobs"][:, 0], a["logprob"].view(-1))
        assert (a["top_logprobs"][:, 1:] <= a["top_logprobs"][:, :-1]).all() and (a["entropy"] > 0).all()


def test_a_step_that_shares_a_cache_takes_its_factors():
    need_gpu()
    layers, rope = _layers(), synth.rotary_tables(64, DIM)
    one = _step(4, 1, 1, 4, rope, layers)
    build = lambda **kw: plans.sparse_decoder_step(layers, DEV, HEADS, KV_HEADS, TOP_K, q_len=11, rope=rope, share=one,
                                                   max_pages=4, cache_bits=4, **kw)
    many = build()
    g = torch.Generator().manual_seed(12)
    for step, n in ((many, 11), (one, 1)):
        step.h.copy_(torch.randn(n, HIDDEN, generator=g))
        before, caches = _state(one), [_held(c) for c in one.caches]
        step.run()
        sync()
        _check_step(step, before, caches, 4, n, rope, layers)
    build(k_factor=KF, v_factor=VF)
    for kw in (dict(k_factor=1.0), dict(v_factor=VF * 2)):
        with pytest.raises(ValueError):
            build(**kw)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("which", ["q", "k"])
def test_layers_that_norm_only_q_or_only_k(bits, which):
    need_gpu()
    layers, rope = _layers(), synth.rotary_tables(64, DIM)
    for L in layers:
        setattr(L, "norm_" + ("k" if which == "q" else "q"), None)
    step = _step(bits, 2, 3, None, rope, layers)
    step.h.copy_(torch.randn(6, HIDDEN, generator=torch.Generator().manual_seed(13)))
    step.seq_lens += 3
    step.run()
    sync()
    pos, cos, sin = np.tile(np.arange(3), 2), ref.f64(rope[0]), ref.f64(rope[1])
    for L, t, cache in zip(layers, step.layers, step.caches):
        rows = lambda n, heads: ref.f64(t[n]).reshape(6, heads, DIM)
        w_q, w_k = (None if w is None else ref.f64(w) for w in (L.norm_q, L.norm_k))
        q, eq, k, ek, _ = serve_ref.head_append(rows("q", HEADS), rows("k", KV_HEADS), w_q, w_k, EPS, 0.0, False, pos,
                                                cos, sin, False)
        ref.check(rows("q_rot", HEADS), q, eq + ref.U16["f16"] * (np.abs(q) + eq) + ref.TINY["f16"], "q")
        held = _held(cache)[0].reshape(2, 4 * PAGE, KV_HEADS, DIM)[:, :3].reshape(6, KV_HEADS, DIM)
        if bits == 4:
            w = [serve_ref.coded(a, e, KF) for a, e in zip(k, ek)]
            ref.check(held, np.stack([a for a, _ in w]), np.stack([b for _, b in w]), "k")
        else:
            ref.check(held, k, ek + ref.U16["f16"] * (np.abs(k) + ek) + ref.TINY["f16"], "k")


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("batch,q_len,pool_pages", [(1, 1, 3), (4, 1, 7), (3, 4, 6), (2, 8, 8)])
def test_idle_sequences(bits, batch, q_len, pool_pages):
    """Sequences that take tokens, rest, end or are refused, in any order, eagerly and by a graph: an idle one keeps its
    pages, its length and its cache, and takes nothing."""
    need_gpu()
    layers, rope = _layers(1), synth.rotary_tables(64, DIM)
    T, M = batch * q_len, batch * q_len
    runs = []
    for graph in (False, True):
        new = torch.full((batch,), q_len, dtype=torch.int32, device=DEV)
        step = _step(bits, batch, q_len, pool_pages, rope, layers, new_lens=new)
        assert step.new_lens is new
        call = step.run
        if graph:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step.run()
            call = captured.replay
        elif batch == 4:                       # another stream, by its handle
            side = torch.cuda.Stream()
            call = lambda: (torch.cuda.synchronize(), step.run(stream=side.cuda_stream))
        r, g, seen = np.random.RandomState(14), torch.Generator().manual_seed(15), []
        for turn in range(30):
            asked = r.choice([q_len, 0, -1], batch, p=[0.6, 0.3, 0.1])
            if turn < 2:
                asked[:] = [0, q_len][turn]
            new.copy_(torch.from_numpy(asked).int())
            step.h.copy_(torch.randn(M, HIDDEN, generator=g))
            before, caches = _state(step), [_held(c) for c in step.caches]
            call()
            sync()
            want = serve_ref.pages(before[0], asked, before[1], before[2], before[3], PAGE, T + 1)
            for got, w in zip(_state(step), want):
                assert np.array_equal(got, w)
            lens, table, starts = want[0], want[1], want[4]
            slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
            for b in np.flatnonzero(asked > 0):
                slots[b * q_len:(b + 1) * q_len] = want[5][starts[b]:starts[b] + q_len]
                pos[b * q_len:(b + 1) * q_len] = want[6][starts[b]:starts[b] + q_len]
            assert np.array_equal(step.slots.cpu().numpy(), slots) and np.array_equal(step.positions.cpu().numpy(), pos)
            grown = lens > np.maximum(before[0], 0)
            assert (grown == ((asked > 0) & (lens != before[0]))).all()
            t, written = step.layers[0], slots >= 0
            rows = lambda n, heads: ref.f64(t[n]).reshape(T, heads, DIM)
            now = _held(step.caches[0])
            for name, held, old, f in (("k", now[0], caches[0][0], KF), ("v", now[1], caches[0][1], VF)):
                flat, was = (c.reshape(-1, KV_HEADS, DIM) for c in (held, old))
                rest = np.setdiff1d(np.arange(len(flat)), slots[written])
                assert np.array_equal(flat[rest], was[rest]), name + ": a place that no token owns"
                if name == "v" and written.any():
                    x = rows("v", KV_HEADS)[written]
                    w = [serve_ref.coded(a, 0 * a, f) for a in x] if bits == 4 else [(a, 0 * a) for a in x]
                    ref.check(flat[slots[written]], np.stack([a for a, _ in w]), np.stack([b for _, b in w]), name)
            args = (rows("q_rot", HEADS), now[0], now[1], table, lens, q_len, DIM ** -0.5)
            ro, _, bo, _ = serve_ref.attention4(*args) if bits == 4 else ref.attention(*args)
            served = np.repeat(grown, q_len)
            ref.check(rows("att", HEADS)[served], ro[served], bo[served], "attention")
            seen.append([step.slots.clone(), step.seq_lens.clone()])
        assert len({tuple(s[1].tolist()) for s in seen}) > 5
        runs.append(seen)
    for a, b in zip(*runs):   # (products of eight rows and more round differently while a graph is captured)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_what_new_lens_may_be():
    need_gpu()
    layers, rope = _layers(1), synth.rotary_tables(64, DIM)
    t = lambda *a, dtype=torch.int32: torch.zeros(a, dtype=dtype, device=DEV)
    for pool, new in ((None, t(2)), (4, t(3)), (4, t(2, dtype=torch.int64)), (4, t(4)[::2])):
        with pytest.raises(ValueError):
            _step(4, 2, 1, pool, rope, layers, new_lens=new)
    one = _step(4, 2, 1, 4, rope, layers)
    many = _step(4, 2, 5, None, rope, layers, share=one, new_lens=t(2))
    many.run()
    sync()
    assert one.seq_lens.tolist() == [0, 0] and one.pool_state.tolist() == [0, 4]
    assert (many.positions == -1).all() and (many.slots == -1).all()
    many.new_lens[1] = 1000                    # more than a step's rows: nothing is read past them
    many.run()
    sync()
    assert one.seq_lens.tolist() == [0, 0]


def test_lengths_on_the_host_are_refused():
    """Their address means nothing on the device."""
    need_gpu()
    layers, rope = _layers(1), synth.rotary_tables(64, DIM)
    with pytest.raises(ValueError):
        _step(4, 2, 1, 4, rope, layers, new_lens=torch.zeros(2, dtype=torch.int32))
    step = _step(4, 2, 1, 4, rope, layers)
    with pytest.raises(ValueError):
        step.end(torch.full((2,), -1, dtype=torch.int32))


def test_a_step_on_the_default_stream_by_its_handle():
    need_gpu()
    new = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    step = _step(4, 2, 1, 4, synth.rotary_tables(64, DIM), _layers(1), new_lens=new)
    step.run(stream=torch.cuda.default_stream().cuda_stream)
    sync()
    assert step.seq_lens.tolist() == [0, 1] and step.slots.tolist() == [-1, 0] and step.positions.tolist() == [-1, 0]
