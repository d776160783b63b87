"""The 8-bit paged cache's calls on batches that contradict their bounds, or that the plan could not serve: what is
refused is refused whole, its error bit is set, and no other sequence sees any of it."""
import random
from types import SimpleNamespace

import pytest
import torch

from block_wise_kv_gb300 import dllm
from kv8_util import PAGE, Batch, assert_attention, cu, ints, plan, random_pools, write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_wise_kv_gb300 import build

    build.build()
    dllm.load()
    torch.cuda.init()


def _desc(H, d):
    return dllm.layer_desc(max(64, H * d), H, d, 1e4)


def _decoded(codes):
    return codes.view(torch.uint8).view(torch.float8_e4m3fn).float().double().cpu()


def _rows(M, heads, d, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(M, heads, d, device="cuda", generator=g).to(torch.bfloat16)


def _written(kv8, n, start, rows, table, cub, served, k, v):
    """The pools after a write in which only the sequences `served` take part."""
    b = SimpleNamespace(n=n, start=start, rows=[r if i in served else 0 for i, r in enumerate(rows)], table=table)
    at = [j for i, r in enumerate(rows) if i in served for j in range(cub[i], cub[i] + r)]
    out = []
    for codes, scale, new in ((kv8.k, kv8.k_scale, k), (kv8.v, kv8.v_scale, v)):
        vals, sc = _decoded(codes), scale.double().cpu()
        write(b, vals, sc, new[at].double().cpu())
        out.append((vals, sc))
    return out


def _assert_pools(kv8, want):
    for (codes, scale), (vals, sc) in zip(((kv8.k, kv8.k_scale), (kv8.v, kv8.v_scale)), want):
        assert torch.equal(scale.double().cpu(), sc)
        assert torch.equal(_decoded(codes), vals)


@pytest.mark.parametrize("start,rows,cub,bound,served", [
    ([80, 89], [10, 11], [0, 10, 21], 20, [0]),                   # more rows than the bound holds
    ([80, 87], [10, 13], [0, 10, 20], 20, [0]),                   # a last block longer than its rows
    ([80, 87, 60], [10, 13, 10], [0, 10, 20, 30], 30, [0, 2]),    # one in the middle: the next one's rows are not its own
    ([80, 80, 60], [10, 30, 10], [0, 10, 10, 20], 20, [0, 2]),    # one that the sums count as none
    ([0, 0], [90, 100], [0, 90, 190], 150, [0]),                  # a prompt that the bound cuts
    ([80, 80], [10, 10], [0, 20, 10], 20, [0]),                   # sums that fall
])
@pytest.mark.parametrize("d", [64, 128])
def test_write_reads_no_row_that_is_not_the_blocks_own(start, rows, cub, bound, served, d):
    """The rows are the front of a larger tensor; what lies behind them is far larger, so that it would show in a scale."""
    b = Batch([100] * len(rows), start, rows, seed=1, cap_rows=bound)
    b.t["cub"].copy_(ints(cub))
    kv8 = random_pools(b.num_pages, 2, d, 3)
    wide = [_rows(max(bound, sum(rows), max(cub)) + 64, 2, d, s) for s in (4, 5)]
    for x in wide:
        x[bound:] = 3000.0
    want = _written(kv8, b.n, start, rows, b.table, cub, served, *wide)
    dllm.dllm_kv8_write(_desc(2, d), b.view.c, wide[0][:bound], wide[1][:bound], kv8.c)
    assert b.bits() == dllm.DLLM_DEVERR_BAD_SHAPE
    _assert_pools(kv8, want)


def test_write_of_a_large_batch_ends_at_the_bound():
    """More sequences than are searched in shared memory, the bound in the middle of one of the last."""
    rows = [3] * 1100
    bound = sum(rows) - 4
    b = Batch([20] * 1100, [14] * 1100, rows, seed=2, cap_rows=bound)
    kv8 = random_pools(b.num_pages, 1, 128, 3)
    wide = [_rows(sum(rows) + 64, 1, 128, s) for s in (4, 5)]
    for x in wide:
        x[bound:] = 3000.0
    want = _written(kv8, b.n, b.start, rows, b.table, cu(rows), range(1098), *wide)
    dllm.dllm_kv8_write(_desc(1, 128), b.view.c, wide[0][:bound], wide[1][:bound], kv8.c)
    assert b.bits() == dllm.DLLM_DEVERR_BAD_SHAPE
    _assert_pools(kv8, want)


def test_write_behind_a_plan_of_more_rows_than_its_bound():
    """The plan flags the batch and leaves its sums whole; the write on the same stream serves what lies within."""
    n, bound, d = [100, 200], 250, 64
    t = dict(n=ints(n), start=ints([0, 0]), rows=ints(n), table=ints([[-1] * 4] * 2), cub=ints([0] * 3), cus=ints([0] * 3),
             held=ints([0, 0]), held_out=ints([0, 0]), err=ints([0]))
    view = dllm.BatchView(t["table"], t["n"], t["start"], t["rows"], t["cub"], t["cus"], bound, 300, 200, 200, t["err"])
    ring = dllm.PageRing.full(8)
    kv8 = random_pools(8, 2, d, 3)
    wide = [_rows(320, 2, d, s) for s in (4, 5)]
    for x in wide:
        x[bound:] = 3000.0
    table = [[0, 1], [2, 3, 4, 5]]
    want = _written(kv8, n, [0, 0], n, table, [0, 100, 300], [0], *wide)
    dllm.dllm_batch_plan(view.c, t["held"], t["held_out"], t["table"], t["cub"], t["cus"], ring.c)
    dllm.dllm_kv8_write(_desc(2, d), view.c, wide[0][:bound], wide[1][:bound], kv8.c)
    assert view.error_bits() == dllm.DLLM_DEVERR_BAD_SHAPE
    assert t["table"].tolist() == [[0, 1, -1, -1], [2, 3, 4, 5]] and PAGE * 6 >= 200
    _assert_pools(kv8, want)


# ------------------------------------------------------------------ the attention
def _attend(view, q, kv8, rows, layout, H, d):
    o = torch.full((rows, H, d), 7.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, H), 7.5, device="cuda")
    ws = dllm.workspace(dllm.dllm_kv8_attention_workspace_size(_desc(H, d), view.c, kv8.c))
    dllm.dllm_kv8_attention(_desc(H, d), view.c, q, kv8.c, o, lse, ws, layout)
    return o, lse


@pytest.mark.parametrize("layout", [dllm.DLLM_ROWS_BLOCK, dllm.DLLM_ROWS_FULL])
@pytest.mark.parametrize("bad", [0, 1, 2])
def test_attention_behind_a_plan_that_counted_a_sequence_as_none(bad, layout):
    """A pages_held that cannot be makes the plan leave its sequence no rows: the attention leaves it out too, and so
    the rows of the next sequence (or, behind the last, of none) are not written twice."""
    n, start, rows, H, kv, d = [150, 100, 300], [100, 20, 290], [10, 30, 7], 4, 2, 64
    b = Batch(n, start, rows, seed=3)
    kv8 = random_pools(b.num_pages, kv, d, 4)
    q = _rows(b.M, H, d, 5)
    held = [(x + PAGE - 1) // PAGE for x in n]
    held[bad] = -3
    t = b.t
    ring = dllm.PageRing(ints([0] * b.num_pages), ints([0, 0]), ints([0, 0]))
    dllm.dllm_batch_plan(b.view.c, ints(held), ints([0] * 3), t["table"], t["cub"], t["cus"], ring.c)
    assert b.bits() == dllm.DLLM_DEVERR_BAD_SHAPE
    left = [r if i != bad else 0 for i, r in enumerate(rows)]
    assert t["cub"].tolist() == cu(left) and t["rows"].tolist() == rows
    b.error.zero_()
    # the packed queries of those that are left
    kept = [j for i, r in enumerate(rows) if i != bad for j in range(cu(rows)[i], cu(rows)[i] + r)]
    qk = q.clone()
    qk[:len(kept)] = q[kept]
    full = layout == dllm.DLLM_ROWS_FULL
    o, lse = _attend(b.view, qk, kv8, b.R if full else b.M, layout, H, d)
    assert b.bits() == dllm.DLLM_DEVERR_BAD_SHAPE
    cus = t["cus"].tolist()
    at = [cus[i] + start[i] + j for i, r in enumerate(left) for j in range(r)] if full else list(range(len(kept)))
    those = SimpleNamespace(n=n, rows=left, table=b.table, M=b.M)
    assert_attention(those, qk, kv8, o[at], lse[at])
    rest = torch.ones(o.shape[0], dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (o[rest] == 7.5).all() and (lse[rest] == 7.5).all()


@pytest.mark.parametrize("cub", [[0, 9, 20], [0, 10, 19], [10, 9, 20], [0, 10, -2147483648]])
def test_attention_refuses_a_block_longer_than_its_rows(cub):
    b = Batch([100, 100], [80, 90], [10, 10], seed=1)
    kv8 = random_pools(b.num_pages, 2, 64, 3)
    q = _rows(b.M, 4, 64, 1)
    b.t["cub"].copy_(ints(cub))
    o, _ = _attend(b.view, q, kv8, b.M, dllm.DLLM_ROWS_BLOCK, 4, 64)
    assert b.bits() == dllm.DLLM_DEVERR_BAD_SHAPE
    for i in (0, 1):
        if cub[i + 1] - cub[i] < 10:
            mine = range(cub[i], cub[i] + 10)
            others = range(cub[1 - i], cub[1 - i] + 10) if cub[2 - i] - cub[1 - i] >= 10 else []
            assert (o[[j for j in mine if j not in others and 0 <= j < 20]] == 7.5).all()


# ------------------------------------------------------------------ a plan that runs short
def test_a_plan_that_runs_short_leaves_no_page_of_another_sequence():
    """The place of a request that has ended is taken by a longer one when no page is free.  Its entries still name the
    pages that went back to the ring and that others hold by now: neither the write nor the attention may follow them."""
    H, kv, d, P = 4, 2, 64, 9
    t = dict(n=ints([250, 60, 190]), start=ints([0, 0, 0]), rows=ints([250, 60, 190]), table=ints([[-1] * 4] * 3),
             cub=ints([0] * 4), cus=ints([0] * 4), err=ints([0]))
    held, held_out, ring = ints([0] * 3), ints([0] * 3), dllm.PageRing.full(P)
    view = dllm.BatchView(t["table"], t["n"], t["start"], t["rows"], t["cub"], t["cus"], 500, 600, 256, 256, t["err"])
    kv8 = random_pools(P, kv, d, 3)

    def step(n, start, rows, seed):
        nonlocal held, held_out, ring
        for key, val in (("n", n), ("start", start), ("rows", rows)):
            t[key].copy_(ints(val))
        before = [x.clone() for x in (kv8.k.view(torch.uint8), kv8.v.view(torch.uint8), kv8.k_scale, kv8.v_scale)]
        k, v, q = _rows(500, kv, d, seed), _rows(500, kv, d, seed + 1), _rows(500, H, d, seed + 2)
        dllm.dllm_batch_plan(view.c, held, held_out, t["table"], t["cub"], t["cus"], ring.c)
        dllm.dllm_kv8_write(_desc(H, d), view.c, k, v, kv8.c)
        o, lse = _attend(view, q, kv8, 500, dllm.DLLM_ROWS_BLOCK, H, d)
        torch.cuda.synchronize()
        held, held_out, ring = held_out, held, ring.swapped()
        return before, k, v, q, o, lse

    step([250, 60, 190], [0, 0, 0], [250, 60, 190], 10)  # four pages, one, three; one left
    assert view.error_bits() == 0
    assert t["table"].tolist() == [[0, 1, 2, 3], [4, -1, -1, -1], [5, 6, 7, -1]]
    step([10, 60, 190], [0, 0, 0], [10, 0, 0], 20)       # the first ends, a short one takes its place: three pages back
    step([10, 256, 190], [10, 60, 190], [0, 196, 0], 30)  # the second grows into them
    assert view.error_bits() == 0
    assert t["table"].tolist() == [[0, 1, 2, 3], [4, 8, 1, 2], [5, 6, 7, -1]]
    # the first wants three pages more and one is free; its entries 1 and 2 name pages of the second
    n, start, rows = [200, 256, 190], [10, 250, 180], [190, 6, 10]
    before, k, v, q, o, lse = step(n, start, rows, 40)
    assert view.error_bits() & dllm.DLLM_DEVERR_NO_PAGES
    assert t["table"].tolist() == [[0, -1, -1, -1], [4, 8, 1, 2], [5, 6, 7, -1]]
    assert held.tolist() == [1, 4, 3]
    table = t["table"].tolist()
    old = dllm.Kv8Cache.of(before[0].view(torch.float8_e4m3fn), before[1].view(torch.float8_e4m3fn), *before[2:])
    want = _written(old, n, start, rows, table, cu(rows), [1, 2], k, v)
    others = [4, 8, 1, 2, 5, 6, 7]
    for (codes, scale), (vals, sc) in zip(((kv8.k, kv8.k_scale), (kv8.v, kv8.v_scale)), want):
        assert torch.equal(scale.double().cpu()[others], sc[others]) and torch.equal(_decoded(codes)[others], vals[others])
    those = SimpleNamespace(n=n[1:], rows=rows[1:], table=table[1:], M=16)
    assert_attention(those, q[190:206], kv8, o[190:206], lse[190:206])
    assert (o[206:] == 7.5).all() and (lse[206:] == 7.5).all()


def test_a_short_plan_called_again_gives_the_same_and_pages_that_come_later_are_taken():
    P = 7
    t = dict(n=ints([100, 256, 64]), rows=ints([1, 1, 1]), start=ints([0, 0, 0]), table=ints([[6, 0, 5, 2], [0, 1, 4, 99], [3, -5, 6, 0]]),
             cub=ints([0] * 4), cus=ints([0] * 4), err=ints([0]))
    ring = dllm.PageRing(ints([5, 2, 0, 0, 0, 0, 3]), ints([6, 3]), ints([0, 0]))  # 3, 5 and 2 are free
    view = dllm.BatchView(t["table"], t["n"], t["start"], t["rows"], t["cub"], t["cus"], 3, 500, 1, 256, t["err"])
    held, out = ints([1, 0, 0]), ints([0] * 3)
    for _ in range(2):
        dllm.dllm_batch_plan(view.c, held, out, t["table"], t["cub"], t["cus"], ring.c)
        # the first has its page; the second is four short, and the third then too; what names no page stays
        assert view.error_bits() == dllm.DLLM_DEVERR_NO_PAGES
        assert t["table"].tolist() == [[6, 3, 5, 2], [-1, -1, -1, 99], [-1, -5, 6, 0]]
        assert out.tolist() == [2, 0, 0] and ring.state_out.tolist() == [0, 2]
    t["n"].copy_(ints([100, 0, 64]))
    t["rows"].copy_(ints([1, 0, 1]))
    ring = ring.swapped()
    dllm.dllm_batch_plan(view.c, out, held, t["table"], t["cub"], t["cus"], ring.c)
    assert held.tolist() == [2, 0, 1] and t["table"].tolist()[2] == [5, -5, 6, 0]


# ------------------------------------------------------------------ places without a request
def _padded(batch=600):
    """A batch of fixed places: those without a request have length 0 and keep a block length and start of before."""
    r = random.Random(7)
    n = [r.choice([0, 0, 40, 200, 333]) for _ in range(batch)]
    rows = [8] * batch
    start = [max(0, x - 8) if x else 77 for x in n]
    return n, start, rows


@pytest.mark.parametrize("batch", [5, 600])
def test_write_and_attention_take_a_length_of_zero_beside_a_block_length(batch):
    n, start, rows = _padded(batch)
    there = [r if x else 0 for x, r in zip(n, rows)]
    b = Batch(n, start, there, seed=1, max_block=8, max_seq=333, max_pages=6)
    b.t["rows"].copy_(ints(rows))
    kv8 = random_pools(b.num_pages, 2, 64, 3)
    k, v, q = _rows(b.M, 2, 64, 4), _rows(b.M, 2, 64, 5), _rows(b.M, 4, 64, 6)
    want = _written(kv8, n, start, there, b.table, cu(there), range(batch), k, v)
    dllm.dllm_kv8_write(_desc(4, 64), b.view.c, k, v, kv8.c)
    assert b.bits() == 0
    _assert_pools(kv8, want)
    o, lse = _attend(b.view, q, kv8, b.M, dllm.DLLM_ROWS_BLOCK, 4, 64)
    assert b.bits() == 0
    assert_attention(b, q, kv8, o, lse)


@pytest.mark.parametrize("batch", [5, 600])
def test_a_plan_takes_a_length_of_zero_beside_a_block_length(batch):
    """Such a place has no rows: nothing is flagged, the pages it held go back, the others are planned."""
    n, start, rows = _padded(batch)
    there = [r if x else 0 for x, r in zip(n, rows)]
    held = [2 if x == 0 else 0 for x in n]
    need = [(x + PAGE - 1) // PAGE for x in n]
    P = sum(held) + sum(need)
    table = [[-1] * 6 for _ in n]
    at = 0
    for b, h in enumerate(held):
        table[b][:h] = range(at, at + h)
        at += h
    ring = list(range(at, P)) + [-1] * at
    M = 8 * batch
    t = dict(table=ints(table), n=ints(n), start=ints(start), rows=ints(rows), cub=ints([0] * (batch + 1)), cus=ints([0] * (batch + 1)),
             err=ints([0]), held=ints(held), out=ints([0] * batch), slot=ints([0] * M), seq=ints([0] * M), pos=ints([0] * M))
    view = dllm.BatchView(t["table"], t["n"], t["start"], t["rows"], t["cub"], t["cus"], M, sum(n), 8, 333, t["err"])
    r = dllm.PageRing(ints(ring), ints([0, P - at]), ints([0, 0]))
    dllm.dllm_batch_plan(view.c, t["held"], t["out"], t["table"], t["cub"], t["cus"], r.c, t["slot"], t["seq"], t["pos"])
    assert view.error_bits() == 0
    now, state, cub, cus, slot, seq, pos, short = plan(n, start, there, held, table, ring, (0, P - at), M)
    assert not short and (t["out"].tolist(), t["cub"].tolist(), t["cus"].tolist()) == (now, cub, cus)
    assert (t["slot"].tolist(), t["seq"].tolist(), t["pos"].tolist()) == (slot, seq, pos)
    assert t["table"].tolist() == table and r.pages.tolist() == ring and r.state_out.tolist() == state
