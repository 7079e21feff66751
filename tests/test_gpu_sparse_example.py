"""The sparse decoder example against a whole model in 64 bits that is fed its tokens."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref
from gpu_util import DEV, need_gpu
from quantized_skinny_gemm_gb300 import synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import sparse_decode  # noqa: E402

HEADS, KV_HEADS, DIM, HIDDEN, INTER, EXPERTS, TOP_K, VOCAB = 6, 2, 64, 256, 96, 8, 3, 512


def _model(layers, embed, lm_head, words):
    """The logits behind each word, one word after the other, in 64 bits."""
    cos, sin = (ref.f64(t) for t in synth.rotary_tables(len(words), DIM))
    rms = lambda h, w: h / np.sqrt((h * h).mean() + 1e-6) * w
    keys, values = ([[] for _ in layers] for _ in range(2))
    logits = []
    for p, word in enumerate(words):
        h = ref.f64(embed[word])
        for i, L in enumerate(layers):
            x = rms(h, ref.f64(L.norm_attn))
            q, k, v = (ref.f64(w) @ x for w in (L.q, L.k, L.v))
            turn = lambda y: ref.rotate(y.reshape(-1, DIM), cos[p], sin[p], DIM, False)[0]
            keys[i].append(turn(k))
            values[i].append(v.reshape(-1, DIM))
            K, V = np.stack(keys[i]), np.stack(values[i])
            att = []
            for n, row in enumerate(turn(q)):
                g = n // (HEADS // KV_HEADS)
                z = K[:, g] @ row * DIM ** -0.5
                e = np.exp(z - z.max())
                att.append(e @ V[:, g] / e.sum())
            h = h + ref.f64(L.o) @ np.concatenate(att)
            x = rms(h, ref.f64(L.norm_mlp))
            z = ref.f64(L.router) @ x
            ids = np.argsort(-z, kind="stable")[:TOP_K]
            w = np.exp(z[ids] - z[ids[0]])
            for e, we in zip(ids, w / w.sum()):
                mat = lambda n: (ref.int4(getattr(L, n)[e].numpy(), ref.f64(L.scales[n][e]), 32) if L.scales
                                 else ref.f64(getattr(L, n)[e]))
                g = mat("gate") @ x
                h = h + we * (mat("down") @ (g / (1 + np.exp(-g)) * (mat("up") @ x)))
        logits.append(ref.f64(lm_head) @ rms(h, 1.0))
    return np.array(logits)


@pytest.mark.gpu
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("prompt", [3, 32, 37])
def test_its_tokens_are_the_models(int4, prompt):
    """Each token must be the model's greedy one, or as good within 0.1 (the logits have
    unit size; thirty roundings to fp16 on the way cost about 0.03).  Where two experts
    tie within a rounding the choice differs and so do the logits: one token in five may."""
    need_gpu()
    layers = synth.sparse_decoder_workload(3, 3, HIDDEN, HEADS, KV_HEADS, DIM, INTER, EXPERTS, int4)
    g = torch.Generator().manual_seed(12)
    embed, lm_head = synth.normal((VOCAB, HIDDEN), 1.0, g), synth.normal((VOCAB, HIDDEN), HIDDEN ** -0.5, g)
    words = torch.randint(0, VOCAB, (prompt,), generator=g)
    tokens = sparse_decode.decode(layers, embed, lm_head, words, 20, HEADS, KV_HEADS, TOP_K, DEV)[0].tolist()
    logits = _model(layers, embed, lm_head, words.tolist() + tokens[:-1])[prompt - 1:]
    gap = logits.max(1) - logits[np.arange(20), tokens]
    assert 0.5 < logits.std() < 2
    assert (gap <= 0.1).sum() >= 16, gap


def test_it_refuses_an_empty_prompt_and_no_tokens():
    layers = synth.sparse_decoder_workload(3, 1, HIDDEN, HEADS, KV_HEADS, DIM, INTER, EXPERTS)
    table = torch.zeros(VOCAB, HIDDEN, dtype=torch.float16)
    for prompt, tokens in ((0, 4), (3, 0)):
        with pytest.raises(ValueError):
            sparse_decode.decode(layers, table, table, torch.zeros(prompt, dtype=torch.int64), tokens, HEADS, KV_HEADS,
                                 TOP_K, torch.device("cpu"))
