"""Greedy decoding with a sparse decoder of random weights: a prompt read in
windows of 16 tokens, then single tokens by one captured CUDA graph.

    python examples/sparse_decode.py [--int4] [--layers 8] [--tokens 64] ...
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_skinny_gemm_gb300 as dg  # noqa: E402
from quantized_skinny_gemm_gb300 import plans, synth  # noqa: E402

WINDOW = 16


def decode(layers, embed, lm_head, prompt, tokens, heads, kv_heads, top_k, device, graph=True):
    """prompt: int64 [P] on the host; embed and lm_head [vocab][hidden]
    fp16.  Returns the `tokens` greedy continuations and the microseconds of a
    step."""
    if not len(prompt) or tokens < 1:
        raise ValueError("a prompt of one token at least, and one token to decode")
    vocab, hidden = embed.shape
    dim = layers[0].q.shape[0] // heads
    total = len(prompt) + tokens
    pages = (total + 63) // 64
    rope = synth.rotary_tables(total, dim)
    E, W = embed.to(device), lm_head.to(device)
    one = plans.sparse_decoder_step(layers, device, heads, kv_heads, top_k, max_pages=pages, rope=rope)
    logits = torch.empty(vocab, dtype=torch.float32, device=device)
    token = torch.empty(1, dtype=torch.int32, device=device)
    head = dg.linear(dg.LINEAR_F16, W, 1, vocab, hidden, x=one.x_out, logits=logits, token=token)
    ws = torch.empty(dg.workspace_bytes([head]), dtype=torch.uint8, device=device)

    window = plans.sparse_decoder_step(layers, device, heads, kv_heads, top_k, q_len=WINDOW, rope=rope, share=one)
    at = 0
    while at < len(prompt):   # a window at a time, the rest one by one
        step, n = (window, WINDOW) if len(prompt) - at >= WINDOW else (one, 1)
        one.seq_lens += n
        step.h.copy_(E[prompt[at:at + n].to(device)])
        step.run()
        at += n
    if step is window:
        one.x_out.copy_(window.x_out[-1:])
    dg.lm_head_argmax(head, ws)

    out = torch.zeros(tokens, dtype=torch.int32, device=device)
    place = torch.zeros(1, dtype=torch.int64, device=device)

    def advance():   # token -> its successor
        out.index_copy_(0, place, token)
        place.add_(1)
        one.seq_lens.add_(1)
        one.h.copy_(E.index_select(0, token))
        one.run()
        dg.lm_head_argmax(head, ws)

    run = advance
    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            advance()
        run = captured.replay
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(tokens):
        run()
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / tokens * 1e6
    dg.check_device_status()
    return out.cpu(), us


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("layers", 8), ("hidden", 2048), ("heads", 16), ("kv-heads", 2), ("head-dim", 128),
                        ("inter", 1024), ("experts", 64), ("top-k", 6), ("vocab", 32768), ("prompt", 200),
                        ("tokens", 64)):
        a.add_argument("--" + name, type=int, default=value)
    a.add_argument("--int4", action="store_true", help="int4 experts")
    a = a.parse_args()
    layers = synth.sparse_decoder_workload(0, a.layers, a.hidden, a.heads, a.kv_heads, a.head_dim, a.inter,
                                           a.experts, a.int4)
    g = synth.generator(1)
    embed = synth.normal((a.vocab, a.hidden), 1.0, g)
    lm_head = synth.normal((a.vocab, a.hidden), a.hidden ** -0.5, g)
    prompt = torch.randint(0, a.vocab, (a.prompt,), generator=g)
    tokens, us = decode(layers, embed, lm_head, prompt, a.tokens, a.heads, a.kv_heads, a.top_k, torch.device("cuda"))
    print("%d layers, %d of %d experts (%s): %.1f us a token" %
          (a.layers, a.top_k, a.experts, "int4" if a.int4 else "fp16", us))
    print("tokens:", " ".join(str(t) for t in tokens.tolist()[:16]), "...")


if __name__ == "__main__":
    main()
