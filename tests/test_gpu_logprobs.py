"""dg_token_logprobs against the definition in 64 bits: rows of every length around a vector
and a tile, ties, masked words, infinities and NaN, odd alignment, parts, graphs."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
import serve_ref
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def run(x, tokens, top_k, scale=1.0, stream=None):
    """x on the device.  logprob, rank, entropy, lse, top_ids, top_logprobs on the host."""
    R = x.shape[0]
    f = lambda *s: torch.full(s, 77.0, dtype=torch.float32, device=DEV)
    i = lambda *s: torch.full(s, 77, dtype=torch.int32, device=DEV)
    out = dict(logprob=f(R), rank=i(R), entropy=f(R), lse=f(R))
    if top_k:
        out.update(top_ids=i(R, top_k), top_logprobs=f(R, top_k))
    td = torch.tensor(tokens, dtype=torch.int32, device=DEV)
    op = dg.logprobs(x, tokens=td, scale=scale, **out)
    need = dg.logprobs_workspace_bytes(op)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV) if need else None
    dg.token_logprobs(op, ws, stream=stream)
    sync()
    return {n: t.cpu().numpy() for n, t in out.items()}


def check(x, tokens, top_k, scale=1.0, what="", got=None):
    got = run(x, tokens, top_k, scale) if got is None else got
    s = float(np.float32(scale))
    lse, lp, H, rank, ids, tops, b_lse, b_lp, b_H = serve_ref.logprobs(ref.f64(x), tokens, top_k, s)
    with np.errstate(over="ignore"):           # what lies past fp32 is infinite there
        lse, lp, tops = (a.astype(np.float32).astype(np.float64) for a in (lse, lp, tops))
    b_lse, b_lp = b_lse + ref.U32 * np.abs(np.nan_to_num(lse, posinf=0, neginf=0)), b_lp * 1.01
    ref.check(got["lse"], lse, b_lse, what + " lse")
    ref.check(got["logprob"], lp, b_lp, what + " logprob")
    ref.check(got["entropy"], H, b_H, what + " entropy")
    assert np.array_equal(got["rank"], rank), what + " rank"
    if top_k:
        assert np.array_equal(got["top_ids"], ids), what + " ids"
        bound = np.maximum(b_lp, b_lse)[:, None] + 4 * ref.U32 * np.abs(np.where(np.isfinite(tops), tops, 0))
        ref.check(got["top_logprobs"], tops, bound, what + " top")


def logits(R, V, ftype, seed, std=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, V, generator=g) * std).to(DT[ftype])


@pytest.mark.parametrize("ftype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V,top_k", [(1, 1), (2, 2), (3, 0), (7, 7), (8, 5), (9, 1), (33, 32), (255, 20), (1000, 5),
                                     (4095, 20), (4096, 32), (4097, 5), (8191, 32), (8193, 20), (32769, 5)])
def test_lengths(ftype, V, top_k):
    """Rows of odd lengths side by side start at every alignment; few rows go in parts."""
    need_gpu()
    x = logits(9, V, ftype, V)
    tokens = np.random.RandomState(V).randint(0, V, 9)
    tokens[0], tokens[1] = 0, V - 1
    check(x.to(DEV), tokens, top_k, what="V %d" % V)


@pytest.mark.parametrize("ftype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,top_k,scale", [(1, 128256, 32, 1.0), (1, 248320, 5, 0.5), (700, 1537, 20, 1.25),
                                             (3, 250001, 20, 2.0), (650, 9000, 1, 1.0)])
def test_wide_and_many_rows(ftype, R, V, top_k, scale):
    need_gpu()
    x = logits(R, V, ftype, R)
    tokens = np.random.RandomState(R).randint(0, V, R)
    check(x.to(DEV), tokens, top_k, scale)


@pytest.mark.parametrize("ftype", ["f16", "f32"])
@pytest.mark.parametrize("R,V", [(2, 30000), (650, 30000)])
@pytest.mark.parametrize("kind", ["equal", "few values", "ascending", "descending", "zeros of both signs", "blocks"])
def test_ties_and_orders(ftype, kind, R, V):
    """Equal logits go by index; every order of the row must find the same words."""
    need_gpu()
    g = torch.Generator().manual_seed(3)
    x = {"equal": lambda: torch.full((V,), 1.5), "few values": lambda: torch.randint(0, 3, (V,), generator=g).float(),
         "ascending": lambda: torch.linspace(-9, 9, V), "descending": lambda: torch.linspace(9, -9, V),
         "zeros of both signs": lambda: torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0),
         "blocks": lambda: torch.arange(V).div(97, rounding_mode="floor").remainder(11).float()}[kind]()
    x = x.to(DT[ftype]).to(DEV).expand(R, V).contiguous()
    tokens = np.random.RandomState(4).randint(0, V, R)
    got = run(x, tokens, 32)
    few = min(R, 4)
    check(x[:few], tokens[:few], 32, what=kind, got={n: t[:few] for n, t in got.items()})
    assert (got["top_ids"] == got["top_ids"][0]).all() and (got["lse"] == got["lse"][0]).all()


@pytest.mark.parametrize("ftype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("parts", [False, True])
def test_masked_words_infinities_and_nan(ftype, parts):
    need_gpu()
    V = 20000
    low = torch.finfo(DT[ftype]).min
    x = logits(12, V, ftype, 5)
    x[0] = -float("inf")                       # nothing left
    x[1] = -float("inf")
    x[1, [5, 19999, 700]] = torch.tensor([1.0, 2.0, 1.0], dtype=x.dtype)   # three words left, 20 asked for
    x[2, ::2] = -float("inf")
    x[3, 3::7] = low                           # masks of the type's lowest value
    x[4] = low
    x[5, 77] = float("nan")
    x[6, 77] = float("inf")
    x[7] = float("nan")
    x[8, [0, V - 1]] = float("nan")
    x[9, 11] = float("inf")
    x[9, 12] = float("inf")
    tokens = np.array([3, 19999, 2, 3, 9, 77, 77, 5, 100, 12, -1, V])
    if not parts:                              # many rows: a row is one CTA's
        x = x.repeat(60, 1)
        tokens = np.tile(tokens, 60)
    got = run(x.to(DEV), tokens, 20)
    check(x[:12].to(DEV), tokens[:12], 20, got={n: t[:12] for n, t in got.items()})
    if not parts:
        for n, t in got.items():
            for i in range(1, 60):
                assert np.array_equal(t[:12], t[12 * i:12 * i + 12], equal_nan=True), n


@pytest.mark.parametrize("ftype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("scale,std", [(1e-20, 3.0), (20.0, 3.0), (1.0, 100.0), (1e30, 1.0), (1.0, 1e-3)])
def test_scales(ftype, scale, std):
    need_gpu()
    x = logits(5, 5000, ftype, 6, std)
    if scale == 1e30:                          # distances of whole logits: one word has all
        x = x.float().round().to(x.dtype)
        x[:, 17] = 50.0
    check(x.to(DEV), [17, 17, 17, 17, 17] if scale == 1e30 else [0, 1, 2, 3, 4999], 3, scale)


@pytest.mark.parametrize("ftype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 3.0])
@pytest.mark.parametrize("V", [5, 3001, 20001])
def test_logits_at_the_ends_of_fp32(ftype, scale, V):
    """Masks of the lowest value around a few words, in every part and at the row's ends; rows of nothing else;
    logits near the largest number."""
    need_gpu()
    low, high = torch.finfo(DT[ftype]).min, torch.finfo(DT[ftype]).max
    x = torch.full((8, V), low, dtype=DT[ftype])
    x[0, V // 2] = 3.0
    x[1, 0], x[1, 1] = 1.0, 0.5
    x[2, V - 1], x[2, V - 2] = 1.0, 0.5
    x[3] = logits(1, V, ftype, 9)[0]
    x[3, :V // 2] = low
    x[4, 1:3] = -float("inf")
    x[5, 2] = high
    x[6, 1], x[6, 3] = high, high
    x[7] = torch.linspace(-3e38, 3e38, V)
    tokens = [V // 2, 1, V - 1, V - 1, 0, 2, 1, V - 1]
    check(x.to(DEV), tokens, min(V, 5), scale)


@pytest.mark.parametrize("ftype", ["f16", "f32"])
def test_strided_rows_and_left_out_outputs(ftype):
    need_gpu()
    V = 3001
    big = torch.full((6, 3500), float("nan"), dtype=DT[ftype])
    big[:, 3:3 + V] = logits(6, V, ftype, 7)
    d = big.to(DEV)
    x = d[:, 3:3 + V]
    tokens = np.arange(6) * 500
    check(x, tokens, 4)
    H = torch.empty(6, dtype=torch.float32, device=DEV)
    op = dg.logprobs(x, entropy=H)
    need = dg.logprobs_workspace_bytes(op)
    dg.token_logprobs(op, torch.empty(need, dtype=torch.uint8, device=DEV) if need else None)
    ids = torch.empty(6, 4, dtype=torch.int32, device=DEV)
    op = dg.logprobs(x, top_ids=ids)
    need = dg.logprobs_workspace_bytes(op)
    dg.token_logprobs(op, torch.empty(need, dtype=torch.uint8, device=DEV) if need else None)
    sync()
    full = run(x, tokens, 4)
    assert np.array_equal(H.cpu().numpy(), full["entropy"]) and np.array_equal(ids.cpu().numpy(), full["top_ids"])


def test_far_rows_streams_graphs_and_repeats():
    need_gpu()
    V = 200000
    far = torch.empty(2, 5 * 10 ** 9, dtype=torch.bfloat16, device=DEV)    # rows more than 2^32 logits apart
    x = far[:, :V]
    x.copy_(logits(2, V, "bf16", 8).to(DEV))
    check(x, [5, 199999], 20)
    td = torch.tensor([5, 199999], dtype=torch.int32, device=DEV)
    lp, rank = torch.empty(2, dtype=torch.float32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    op = dg.logprobs(x, tokens=td, logprob=lp, rank=rank)
    ws = torch.empty(dg.logprobs_workspace_bytes(op), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.token_logprobs(op, ws)
    side = torch.cuda.Stream()
    for seed in (9, 10):
        x.copy_(logits(2, V, "bf16", seed).to(DEV))
        graph.replay()
        sync()
        got = run(x, [5, 199999], 0, stream=side)
        assert np.array_equal(lp.cpu().numpy(), got["logprob"]) and np.array_equal(rank.cpu().numpy(), got["rank"])
        check(x, [5, 199999], 0, got=got)


@pytest.mark.parametrize("ftype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,V", [(70, 20011), (640, 8300)])
@pytest.mark.parametrize("wide", [False, True])
def test_ranks_between_neighbouring_numbers(ftype, R, V, wide):
    """Zeros of both signs, the smallest and largest numbers and their neighbours, with tokens around the
    ends of vectors and tiles: a rank counts equal ones before the token, and no other number."""
    need_gpu()
    it = {"f16": torch.int16, "bf16": torch.int16, "f32": torch.int32}[ftype]
    one = int(torch.tensor(1.0, dtype=DT[ftype]).view(it))
    few = [0, 1, 2, one - 1, one, one + 1]
    if wide:
        top = int(torch.tensor(torch.finfo(DT[ftype]).max, dtype=DT[ftype]).view(it))
        few += [top - 1, top, top + 1]         # the last: infinity, below only with a sign
    sign = 1 << (15 if it == torch.int16 else 31)
    all_ = [v - 2 * sign for v in (sign + f for f in few)] + [f for f in few if not wide or f != top + 1]
    g = torch.Generator().manual_seed(12)
    bits = torch.tensor(all_, dtype=torch.int64)[torch.randint(0, len(all_), (4, V), generator=g)].to(it)
    x = bits.view(DT[ftype]).repeat(R // 4, 1).contiguous()
    R = x.shape[0]
    tokens = np.concatenate([np.arange(24), 4090 + np.arange(12), 8184 + np.arange(16), V - 1 - np.arange(8)])
    tokens = np.resize(np.repeat(tokens, 4), R)
    got = run(x.to(DEV), tokens, 0)
    for r in range(R):
        row = ref.f64(x[r])
        t = tokens[r]
        assert got["rank"][r] == (row > row[t]).sum() + (row[:t] == row[t]).sum(), (r, t, row[t])


@pytest.mark.parametrize("ftype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-38, 1e-31, 2.5e-31, 1e-20])
@pytest.mark.parametrize("V", [7, 30001])
def test_high_temperatures(ftype, scale, V):
    """Every finite logit weighs the same; masked ones nothing."""
    need_gpu()
    x = logits(5, V, ftype, 9)
    x[1, ::3] = -float("inf")
    x[2] = -float("inf")
    x[3, ::2] = torch.finfo(DT[ftype]).min
    x[4] = -float("inf")
    x[4, 5] = 2.0
    check(x.to(DEV), [0, 1, 2, 3, 5], 3, scale)


@pytest.mark.parametrize("ftype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,V,top_k", [(1217, 20000, 5), (1260, 9001, 32), (763, 9001, 0), (800, 30000, 20), (2500, 5000, 1)])
def test_whole_rows_and_rows_in_parts_in_one_call(ftype, R, V, top_k):
    """Rows behind the last full round go in parts: the same rows there and before have the same words and ranks."""
    need_gpu()
    x = logits(17, V, ftype, R)
    x[3, ::2] = -float("inf")
    x[5] = x[5].clamp(-1, 1)                   # ties
    x[7, V // 2] = float("nan")
    tokens = np.random.RandomState(R).randint(-1, V + 1, 17)
    tokens[3] = 1
    n = -(-R // 17)
    got = run(x.repeat(n, 1)[:R].to(DEV), np.tile(tokens, n)[:R], top_k, 0.75)
    check(x.to(DEV), tokens, top_k, 0.75, "first", {k: t[:17] for k, t in got.items()})
    at = (R - 17) // 17 * 17
    check(x.to(DEV), tokens, top_k, 0.75, "last whole", {k: t[at:at + 17] for k, t in got.items()})
    last = np.arange(R - 17, R) % 17
    check(x[last].to(DEV), tokens[last], top_k, 0.75, "last", {k: t[R - 17:] for k, t in got.items()})
    for k in ("rank", "top_ids")[:2 if top_k else 1]:
        assert np.array_equal(got[k], np.concatenate([got[k][:17]] * n)[:R]), k


@pytest.mark.parametrize("ftype", ["f16", "f32"])
@pytest.mark.parametrize("V", [129, 260, 517, 1030, 2053])
def test_ranks_of_many_short_rows(ftype, V):
    """Rows of about as many vectors as a CTA has threads, a token that all others come before: the warps reach the
    row's end at different times, some with nothing of it, and none of their counts may be lost."""
    need_gpu()
    R = 6000
    x = logits(1, V, ftype, V).repeat(R, 1)
    tokens = np.random.RandomState(V).randint(0, V, R)
    x[torch.arange(R), torch.from_numpy(tokens)] = -60.0
    for _ in range(3):
        got = run(x.to(DEV), tokens, 0)
        assert (got["rank"] == V - 1).all()


BORDER = 2 ** 22 * float(np.log(2))            # of z, where its size in powers of two passes 2^22


@pytest.mark.parametrize("ftype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("side", [-1, 1])
@pytest.mark.parametrize("V,lower", [(5, 1.0), (5, 40.0), (129, 1.0), (130, 6.0), (3001, 3.0), (20001, 1.0), (20001, 9.0)])
def test_best_logits_around_a_border_of_the_arithmetic(ftype, side, V, lower):
    """The best z on both sides of +-2^22 powers of two, the others a little lower: no weight is lost, and sums and
    log probabilities count from the same number, in rows at every alignment, whole and in parts."""
    need_gpu()
    past = [-300.0, -90.0, -7.0, -1.0, 0.0, 0.25, 1.0, 5.0, 30.0, 60.0, 80.0, 86.0, 87.0, 88.0, 89.0, 95.0, 128.0, 400.0]
    if ftype == "f32":                         # steps of 0.25 around 2907270
        best, scale, step = [side * BORDER - p for p in past], 1.0, lower
    else:                                      # 33 is the border; steps of 1 / 32 (f16) and 1 / 4 (bf16) there
        best, scale, step = [side * 33.0 - p / 1024 for p in past], BORDER / 33.0, lower * 2 ** -7
        if ftype == "bf16":
            step = 0.25
    R = len(best)
    x = torch.empty(R, V)
    g = torch.Generator().manual_seed(V)
    for r, b in enumerate(best):
        x[r] = round(b * 64) / 64 - step * torch.randint(1, 3, (V,), generator=g)
        x[r, (r * 37) % V] = round(b * 64) / 64
    x = x.to(DT[ftype])
    x[3, V // 2] = 1.0 if side < 0 else -1.0   # one word far above the rest, or below
    x[7, 0] = torch.finfo(DT[ftype]).min       # and a masked one
    tokens = np.arange(R) * 37 % V
    tokens[::2] = (tokens[::2] + 1) % V
    check(x.to(DEV), tokens, min(V, 4), scale)
    if V == 5:                                 # every row a CTA's
        many = x.repeat(45, 1)
        got = run(many.to(DEV), np.tile(tokens, 45), 4, scale)
        check(x.to(DEV), tokens, 4, scale, "whole", {n: t[:R] for n, t in got.items()})


@pytest.mark.parametrize("where", ["first", "last", "spread"])
@pytest.mark.parametrize("scale", [1.0, 1000.0, 1e5])
@pytest.mark.parametrize("V", [20003, 60001])
def test_parts_on_both_sides_of_the_border(where, scale, V):
    """The parts of one row lie on different sides of the border, with weights of about the same size."""
    need_gpu()
    for side in (-1, 1):
        x = torch.full((3, V), (side * BORDER - 60.0) / scale)
        near = {"first": np.arange(0, V // 3), "last": np.arange(V - V // 3, V), "spread": np.arange(0, V, 5000)}[where]
        for r, over in enumerate((0.5, 3.0, 20.0)):
            x[r] = x[r] + 60.0 / scale - 2.0 / scale
            x[r, near] += over / scale
        tokens = [0, V - 1, V // 2]
        check(x.to(DEV), tokens, 5, scale)


@pytest.mark.parametrize("ftype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-30, 3e-25, 0.5])
@pytest.mark.parametrize("V", [6, 20001])
def test_differences_past_fp32_of_logits_inside_it(ftype, scale, V):
    """Two logits 6e38 apart: their difference is no number of fp32, a small multiple of it is."""
    need_gpu()
    x = torch.full((3, V), 2.5e38, dtype=DT[ftype])
    x[0, 1], x[0, V - 1] = 3e38, -3e38
    x[1] = -3e38
    x[1, V // 2] = 3e38
    x[2, 0], x[2, 3] = -2e38, 1.5e38
    check(x.to(DEV), [V - 1, 0, 0], 6, scale)
