"""dg_assign_pages against the rules, one sequence after the other on the host."""
import numpy as np
import pytest
import torch

import quantized_skinny_gemm_gb300 as dg
import serve_ref
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
I32 = torch.int32


def setup(B, page, len_max, new, seed, free=None, spare=3, first=None):
    """lens, table, pool, state on the host: pages in no order, the queue begun anywhere."""
    r = np.random.RandomState(seed)
    lens = r.randint(0, len_max + 1, B).astype(np.int32)
    lens[r.rand(B) < 0.2] = 0
    held = -(-lens.astype(np.int64) // page)
    width = int(-(-(len_max + max(int(new.max()), 0)) // page)) + 1
    need = int((-(-(lens.astype(np.int64) + np.maximum(new, 0)) // page) - held).sum())
    size = int(held.sum()) + need + spare
    order = r.permutation(size).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = size - at if free is None else min(free, size - at)
    first = int(r.randint(0, size)) if first is None else first
    pool = np.full(size, -9, np.int32)
    pool[(first + np.arange(free)) % size] = order[at:at + free]
    return lens, table, pool, np.array([first, free], np.int32)


def run(lens, new, table, pool, state, page, tokens, in_place=False, uniform=None, stream=None, extra=0):
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    ld, nd, pd, sd = dev(lens), dev(new.astype(np.int32)), dev(pool), dev(state)
    wide = torch.full((len(lens), table.shape[1] + extra), -7, dtype=I32, device=DEV)
    td = wide[:, :table.shape[1]]
    td.copy_(dev(table))
    lo = ld if in_place else torch.full_like(ld, 77)
    so = sd if in_place else torch.full_like(sd, 77)
    starts = torch.full((len(lens) + 1,), 77, dtype=I32, device=DEV)
    slots = torch.full((tokens,), 77, dtype=torch.int64, device=DEV) if tokens else None
    positions = torch.full((tokens,), 77, dtype=I32, device=DEV) if tokens else None
    op = dg.page_plan(ld, td, pd, sd, page, new_lens=nd if uniform is None else None, new_len=uniform or 0, lens_out=lo,
                      pool_state_out=so, starts=starts, slots=slots, positions=positions)
    need = dg.pages_workspace_bytes(op)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV) if need else None
    dg.assign_pages(op, ws, stream=stream)
    sync()
    assert (wide[:, table.shape[1]:] == -7).all()
    if not in_place:
        assert np.array_equal(ld.cpu().numpy(), lens) and np.array_equal(sd.cpu().numpy(), state)
    n = lambda t: None if t is None else t.cpu().numpy()
    return n(lo), n(td), n(pd), n(so), n(starts), n(slots), n(positions)


def check(got, want):
    for name, g, w in zip(("lens", "table", "pool", "state", "starts", "slots", "positions"), got, want):
        assert g is None or np.array_equal(g.astype(np.int64), w.astype(np.int64)), name


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,len_max,news,ended,free", [
    (1, 16, 40, 1, 0, None), (1, 1, 0, 5, 0, None), (7, 16, 100, 1, 0, None), (64, 16, 500, 8, 10, None),
    (33, 7, 64, 20, 30, 4), (1024, 16, 300, 1, 5, 11), (1025, 16, 300, 3, 5, 100), (300, 64, 3000, 700, 3, 900),
    (5000, 16, 100, 2, 20, None), (4097, 24, 60, 9, 0, 0), (128, 256, 4000, 1, 0, 3), (50, 16, 200, 40, 100, None),
])
def test_growth_ends_and_a_short_pool(B, page, len_max, news, ended, free, in_place):
    need_gpu()
    r = np.random.RandomState(B)
    new = r.randint(0 if B > 1 else 1, news + 1, B)
    new[r.rand(B) * 100 < ended] = -1 - r.randint(0, 3)
    lens, table, pool, state = setup(B, page, len_max, new, B + 1, free)
    tokens = int(np.maximum(new, 0).sum()) + 5
    check(run(lens, new, table, pool, state, page, tokens, in_place, extra=2),
          serve_ref.pages(lens, new, table, pool, state, page, tokens))


@pytest.mark.parametrize("B", [40, 2000])
def test_a_map_that_is_too_short_and_a_table_that_is(B):
    """Who does not fit is left out, and those behind it are served if they fit."""
    need_gpu()
    r = np.random.RandomState(3)
    new = r.randint(0, 30, B)
    lens, table, pool, state = setup(B, 16, 200, new, 4)
    for tokens in (1, int(new[:B // 2].sum()), int(new.sum()) - 1, int(new.sum())):
        check(run(lens, new, table, pool, state, 16, tokens),
              serve_ref.pages(lens, new, table, pool, state, 16, tokens))
    narrow = np.ascontiguousarray(table[:, :8])            # 128 positions; longer ones hold more than they may
    check(run(lens, new, narrow, pool, state, 16, 4000 if B == 40 else 40000),
          serve_ref.pages(lens, new, narrow, pool, state, 16, 4000 if B == 40 else 40000))


@pytest.mark.parametrize("B", [3, 3000])
def test_without_a_map_and_one_length_for_all(B):
    need_gpu()
    new = np.full(B, 4)
    lens, table, pool, state = setup(B, 16, 99, new, 5, free=B // 2 + 1)
    check(run(lens, new, table, pool, state, 16, 0, uniform=4),
          serve_ref.pages(lens, new, table, pool, state, 16, 0))


def test_odd_states():
    """Lengths below zero hold nothing, a count past the queue's size or below zero is the nearest
    right one, tables that name no page give no slot, and a full queue takes nothing back."""
    need_gpu()
    new = np.array([3, 3, 0, -1, 20, 2])
    lens = np.array([-4, 17, 5, 40, 2 ** 31 - 10, -2 ** 31], np.int32)
    table = np.arange(60, dtype=np.int32).reshape(6, 10) + 100
    table[1, 1] = -1
    pool = np.arange(12, dtype=np.int32)
    for state in ([3, 12], [3, 99], [0, -5], [11, 4]):
        state = np.array(state, np.int32)
        kept = np.array([state[0], min(max(state[1], 0), 12)])
        want = serve_ref.pages(np.maximum(lens, -1), new, table, pool, kept, 16, 40)
        lo = want[0]
        lo[0] = -4 if lo[0] < 0 else lo[0]
        lo[5] = -2 ** 31 if lo[5] < 0 else lo[5]
        check(run(lens, new, table, pool, state, 16, 40), want)


def test_a_run_of_steps_in_a_graph():
    """Thirty steps of joining, growing and ending sequences: nobody shares a page, none is lost."""
    need_gpu()
    B, page, width, N, tokens = 24, 4, 30, 200, 24 * 9
    ld = torch.zeros(B, dtype=I32, device=DEV)
    nd = torch.zeros(B, dtype=I32, device=DEV)
    td = torch.full((B, width), -1, dtype=I32, device=DEV)
    pd = torch.randperm(N, generator=torch.Generator().manual_seed(6)).int().to(DEV)
    sd = torch.tensor([150, N], dtype=I32, device=DEV)
    starts = torch.empty(B + 1, dtype=I32, device=DEV)
    slots, positions = torch.empty(tokens, dtype=torch.int64, device=DEV), torch.empty(tokens, dtype=I32, device=DEV)
    op = dg.page_plan(ld, td, pd, sd, page, new_lens=nd, starts=starts, slots=slots, positions=positions)
    assert dg.pages_workspace_bytes(op) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.assign_pages(op)
    r = np.random.RandomState(7)
    state = [ld, td, pd, sd]
    for step in range(30):
        new = r.randint(0, 10, B)
        new[r.rand(B) < 0.1] = -1
        nd.copy_(torch.from_numpy(new.astype(np.int32)))
        lens, table, pool, st = (t.cpu().numpy().copy() for t in state)
        want = serve_ref.pages(lens, new, table, pool, st, page, tokens)
        graph.replay()
        sync()
        check([t.cpu().numpy() for t in state + [starts, slots, positions]], want)
        lens, table, pool, st = (t.cpu().numpy() for t in state)
        used = [p for b in range(B) for p in table[b, :-(-lens[b] // page)]]
        free = [pool[(st[0] + i) % N] for i in range(st[1])]
        assert sorted(used + free) == list(range(N)), "step %d" % step
    assert (lens > 0).any()


def test_another_stream():
    need_gpu()
    new = np.full(2000, 2)
    lens, table, pool, state = setup(2000, 16, 99, new, 8)
    side = torch.cuda.Stream()
    check(run(lens, new, table, pool, state, 16, 4000, stream=side),
          serve_ref.pages(lens, new, table, pool, state, 16, 4000))


@pytest.mark.parametrize("B,len_max", [(1, 40000), (5, 9001), (90, 1500), (1024, 200), (1500, 60)])
@pytest.mark.parametrize("page", [1, 16])
def test_long_sequences_that_end_together(B, len_max, page):
    """More pages come back than the launch has threads, in runs that start and end inside a row."""
    need_gpu()
    r = np.random.RandomState(6)
    new = np.where(r.rand(B) < 0.8, -1, r.randint(0, 4, B))
    new[0] = -1
    lens, table, pool, state = setup(B, page, len_max, new, 7)
    tokens = int(np.maximum(new, 0).sum()) + 3
    check(run(lens, new, table, pool, state, page, tokens), serve_ref.pages(lens, new, table, pool, state, page, tokens))


@pytest.mark.parametrize("kind", ["mixed", "one", "tiny", "few"])
def test_maps_of_many_tokens(kind):
    """Runs of several tokens a lane: sequences of none, of one and of thousands side by side, some not served."""
    need_gpu()
    r = np.random.RandomState(8)
    new = {"mixed": lambda: np.where(r.rand(3000) < 0.4, 0, np.where(r.rand(3000) < 0.6, r.randint(1, 4, 3000),
                                                                     r.randint(500, 2500, 3000))),
           "one": lambda: np.array([0, 0, 650000, 0]), "tiny": lambda: r.randint(0, 2, 900000 // 4) * 3,
           "few": lambda: np.array([1, 300001, 0, 255, 257, 256, 1, 1, 200000, 0])}[kind]()
    lens, table, pool, state = setup(len(new), 16, 60, new, 9)
    total = int(new.sum())
    assert total > 330000
    for tokens in (total, total - 1000, total + 70):
        check(run(lens, new, table, pool, state, 16, tokens), serve_ref.pages(lens, new, table, pool, state, 16, tokens))
