"""The 8-bit paged cache on the GPU: the batch plan, the quantising writes and the attention, each against a plain 64-bit
implementation (tests/kv8_util.py), and a run of them together."""
import random

import numpy as np
import pytest
import torch

from block_wise_kv_gb300 import dllm
from block_wise_kv_gb300.inputs import Workload, make_config
from block_wise_kv_gb300.step import LayerStep, block_rows_of, full_rows_of
from kv8_util import G, PAGE, Batch, assert_attention, attention, ints, plan, random_pools, values, write

pytestmark = pytest.mark.gpu
NAN_CODE = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_wise_kv_gb300 import build

    build.build()
    dllm.load()
    torch.cuda.init()


def _desc(H, d):
    return dllm.layer_desc(max(64, H * d), H, d, 1e4)


# ------------------------------------------------------------------ the plan
class Plan:
    def __init__(self, n, start, rows, held, total, free, seed=0, cap=None, head=None, max_seq=None):
        r = random.Random(seed)
        ids = list(range(total))
        r.shuffle(ids)
        self.wide = max([1] + [(x + 63) // 64 for x in n] + list(held) + [((max_seq or 1) + 63) // 64])
        self.table = [[-7] * self.wide for _ in n]
        at = 0
        for b, h in enumerate(held):
            self.table[b][:h] = ids[at:at + h]
            at += h
        self.head = r.randrange(total) if head is None else head
        self.ring = [-9] * total
        for k in range(free):
            self.ring[(self.head + k) % total] = ids[at + k]
        self.free = free
        self.n, self.start, self.rows, self.held = n, start, rows, held
        self.cap = sum(rows) if cap is None else cap
        d = self.d = dict(n=ints(n), start=ints(start), rows=ints(rows), held=ints(held), table=ints(self.table).view(len(n), self.wide),
                          ring=ints(self.ring), state=ints([self.head, free]), state_out=ints([-5, -5]),
                          held_out=ints([-5] * len(n)), cub=ints([-5] * (len(n) + 1)), cus=ints([-5] * (len(n) + 1)),
                          slot=ints([-5] * self.cap), seq=ints([-5] * self.cap), pos=ints([-5] * self.cap), err=ints([0]))
        self.view = dllm.BatchView(d["table"], d["n"], d["start"], d["rows"], d["cub"], d["cus"], self.cap, max(1, sum(n)),
                                   max([1] + rows), max_seq or max([1] + n), d["err"])

    def call(self):
        d = self.d
        ring = dllm.PageRing(d["ring"], d["state"], d["state_out"])
        dllm.dllm_batch_plan(self.view.c, d["held"], d["held_out"], d["table"], d["cub"], d["cus"], ring.c, d["slot"], d["seq"],
                             d["pos"])

    def check(self):
        torch.cuda.synchronize()
        table, ring = [list(x) for x in self.table], list(self.ring)
        now, state, cub, cus, slot, seq, pos, short = plan(self.n, self.start, self.rows, self.held, table, ring,
                                                           (self.head, self.free), self.cap)
        d = {k: v.tolist() for k, v in self.d.items()}
        assert d["held_out"] == now and d["state_out"] == state and d["cub"] == cub and d["cus"] == cus
        assert d["table"] == table and d["ring"] == ring
        assert d["slot"] == slot and d["seq"] == seq and d["pos"] == pos
        assert d["err"][0] == (dllm.DLLM_DEVERR_NO_PAGES if short else 0)


@pytest.mark.parametrize("n,start,rows,held,free", [
    ([1], [0], [1], [0], 1),
    ([64], [0], [64], [0], 3),
    ([65], [64], [1], [1], 1),
    ([0], [0], [0], [2], 1),          # ends: both pages go back
    ([0, 0, 0], [0, 0, 0], [0, 0, 0], [0, 0, 0], 2),
    ([130, 0, 64, 1], [98, 0, 0, 0], [32, 0, 64, 1], [2, 3, 4, 0], 2),
    ([300, 10, 70], [0, 0, 6], [300, 10, 64], [0, 0, 1], 4),  # the first asks for more than is free
    ([64, 640, 64], [0, 0, 0], [1, 1, 1], [0, 0, 0], 5),      # the second does, and the third then too
])
def test_plan_small(n, start, rows, held, free):
    p = Plan(n, start, rows, held, sum(held) + free + 2, free, cap=sum(rows) + 3)
    p.call()
    p.check()
    p.call()  # the call reads only what it does not write: the same again
    p.check()


@pytest.mark.parametrize("batch,longest,short", [(7, 300, 1.0), (200, 5000, 1.0), (1024, 400, 0.7), (1025, 130, 1.0),
                                                 (2500, 700, 1.0), (3, 200000, 1.0)])
def test_plan_ragged(batch, longest, short):
    r = random.Random(batch)
    n = [r.choice([0, r.randint(1, longest), r.randint(1, longest)]) for _ in range(batch)]
    rows = [r.randint(0, min(x, r.choice([1, 64, longest]))) for x in n]
    start = [r.randint(0, x - k) for x, k in zip(n, rows)]
    held = [max(0, (x + 63) // 64 + r.randint(-3, 2)) for x in n]
    asked = sum(max(0, (x + 63) // 64 - h) for x, h in zip(n, held))
    free = int(asked * short)
    p = Plan(n, start, rows, held, sum(held) + free + 1, free, seed=batch, cap=sum(rows) + 17)
    p.call()
    p.check()


def test_plan_of_no_sequences():
    p = Plan([], [], [], [], 4, 3, cap=5)
    p.call()
    p.check()


def test_plan_without_row_maps_and_rows_beyond_the_bound():
    p = Plan([100, 200], [0, 0], [100, 200], [0, 0], 10, 8)
    d = p.d
    ring = dllm.PageRing(d["ring"], d["state"], d["state_out"])
    dllm.dllm_batch_plan(p.view.c, d["held"], d["held_out"], d["table"], d["cub"], d["cus"], ring.c)
    assert d["held_out"].tolist() == [2, 4] and d["slot"].tolist() == [-5] * 300
    p.view.c.total_block_rows = 250
    dllm.dllm_batch_plan(p.view.c, d["held"], d["held_out"], d["table"], d["cub"], d["cus"], ring.c, d["slot"])
    assert d["slot"].tolist()[250:] == [-5] * 50 and min(d["slot"].tolist()[:250]) >= 0
    assert p.view.error_bits() == dllm.DLLM_DEVERR_BAD_SHAPE


@pytest.mark.parametrize("change,bit", [
    (dict(n=[-1, 70]), 4), (dict(n=[1 << 30, 70]), 4), (dict(held=[-3, 0]), 4), (dict(held=[1 << 30, 0]), 4),
    (dict(start=[60, 0]), 4), (dict(start=[-1, 0]), 4), (dict(rows=[65, 70]), 4), (dict(rows=[-1, 70]), 4),
    (dict(state=[99, 2]), 4 | 16), (dict(state=[0, 99]), 4 | 16), (dict(state=[-1, 2]), 4 | 16), (dict(ring=[77] * 9), 2)])
def test_plan_refuses_what_contradicts_the_bounds(change, bit):
    p = Plan([64, 70], [0, 0], [30, 70], [0, 0], 9, 5, cap=200)
    for k, v in change.items():
        p.d[k].copy_(ints(v))
    p.call()
    assert p.view.error_bits() == bit
    d = {k: v.tolist() for k, v in p.d.items()}
    if bit == 4 and "held" not in change:
        assert d["seq"].count(1) == 70  # the other sequence is planned
        assert [x for x, s in zip(d["slot"], d["seq"]) if s == 1][0] >= 0
    if "held" in change or "n" in change:
        assert d["held_out"][0] == d["held"][0] and 0 not in d["seq"]
    assert all(-1 <= x < 9 * 64 for x in d["slot"])


def test_plan_refuses_ids_that_are_no_pages_in_the_table():
    p = Plan([0, 10], [0, 0], [0, 10], [2, 1], 9, 3)
    p.d["table"].copy_(ints([[50, 3], [-4, 0]]))
    p.call()
    assert p.view.error_bits() == dllm.DLLM_DEVERR_BAD_PAGE
    assert p.d["slot"].tolist() == [-1] * 10
    assert [p.d["ring"].tolist()[(p.head + 3 + k) % 9] for k in range(2)] == [-1, 3]


def test_plan_many_steps_keeps_every_page_once():
    r = random.Random(1)
    P, batch = 60, 12
    ring = dllm.PageRing.full(P)
    held, held_out = ints([0] * batch), ints([0] * batch)
    table, cub, cus, err = ints([[0] * 8] * batch), ints([0] * (batch + 1)), ints([0] * (batch + 1)), ints([0])
    n = [0] * batch
    view = dllm.BatchView(table, ints(n), ints(n), ints(n), cub, cus, 100, 8 * 64 * batch, 64, 512, err)
    for _ in range(40):
        n = [r.choice([0, min(512, x + r.randint(0, 64)), min(512, x + 1)]) if r.random() < 0.5 else x for x in n]
        view.tensors[1].copy_(ints(n))
        dllm.dllm_batch_plan(view.c, held, held_out, table, cub, cus, ring.c)
        held, held_out, ring = held_out, held, ring.swapped()
        h, t = held.tolist(), table.tolist()
        head, count = ring.state.tolist()
        free = [ring.pages.tolist()[(head + k) % P] for k in range(count)]
        assert sorted(free + [i for b in range(batch) for i in t[b][:h[b]]]) == list(range(P))
        assert all(x <= (y + 63) // 64 or err.item() == 0 for x, y in zip(h, n))


# ------------------------------------------------------------------ the writes
def _rows(M, kv, d, seed, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return [(torch.randn(M, kv, d, device="cuda", generator=g) * size *
             torch.exp(torch.randn(1, kv, d, device="cuda", generator=g))).to(torch.bfloat16) for _ in range(2)]


def _expected(b, kv8, k_new, v_new):
    out = []
    for codes, scale, new in ((kv8.k, kv8.k_scale, k_new), (kv8.v, kv8.v_scale, v_new)):
        vals = codes.view(torch.uint8).view(torch.float8_e4m3fn).float().double().cpu()
        sc = scale.double().cpu()
        write(b, vals, sc, new.double().cpu())
        out.append((vals, sc))
    return out


def _assert_written(kv8, want):
    for (codes, scale), (vals, sc) in zip(((kv8.k, kv8.k_scale), (kv8.v, kv8.v_scale)), want):
        assert torch.equal(scale.double().cpu(), sc)
        assert torch.equal(codes.view(torch.uint8).view(torch.float8_e4m3fn).float().double().cpu(), vals)


WRITES = [
    # lengths, block starts, block lengths, heads, d
    ([1], [0], [1], 1, 128),
    ([320], [32], [32], 2, 64),
    ([17, 64, 65], [16, 63, 64], [1, 1, 1], 3, 128),
    ([100, 7, 0, 40, 0], [13, 0, 0, 39, 0], [50, 7, 0, 1, 0], 2, 128),
    ([130, 30], [0, 3], [130, 20], 5, 64),           # a whole prompt; a block inside one group and the next
    ([20, 33], [1, 0], [3, 33], 4, 128),             # rows of the group on both sides stay
    ([300] * 9, list(range(0, 270, 30)), [30] * 9, 2, 64),
]


@pytest.mark.parametrize("n,start,rows,kv,d", WRITES)
@pytest.mark.parametrize("size", [0.01, 1.0, 100.0])
def test_write_rows(n, start, rows, kv, d, size):
    b = Batch(n, start, rows, seed=len(n))
    kv8 = random_pools(b.num_pages, kv, d, 3)
    k, v = _rows(b.M, kv, d, 4, size)
    want = _expected(b, kv8, k, v)
    dllm.dllm_kv8_write(_desc(2 * kv, d), b.view.c, k, v, kv8.c)
    assert b.bits() == 0
    _assert_written(kv8, want)
    dllm.dllm_kv8_write(_desc(2 * kv, d), b.view.c, k, v, kv8.c)  # the scales have what they need: the same again
    _assert_written(kv8, want)


def test_write_takes_the_wide_slices_too():
    n = [700, 1, 2000, 64, 333]
    b = Batch(n, [5, 0, 0, 0, 100], [690, 1, 2000, 64, 233], seed=1)
    kv8 = random_pools(b.num_pages, 26, 64, 3)
    k, v = _rows(b.M, 26, 64, 4)
    want = _expected(b, kv8, k, v)
    dllm.dllm_kv8_write(_desc(26, 64), b.view.c, k, v, kv8.c)
    assert b.bits() == 0
    _assert_written(kv8, want)


def test_write_large_batch_of_single_tokens():
    r = random.Random(5)
    n = [r.randint(0, 90) for _ in range(1500)]
    b = Batch(n, [max(0, x - 1) for x in n], [min(1, x) for x in n], cap_rows=1500)
    kv8 = random_pools(b.num_pages, 1, 128, 3)
    k, v = _rows(1500, 1, 128, 4)
    want = _expected(b, kv8, k, v)
    dllm.dllm_kv8_write(_desc(1, 128), b.view.c, k, v, kv8.c)
    assert b.bits() == 0
    _assert_written(kv8, want)


def test_write_token_by_token():
    """Appending grows scales step by step: the codes stay within what one write of each growth leaves."""
    kv8 = random_pools(3, 2, 64, 1)
    k, v = _rows(40, 2, 64, 2)
    k, v = [(x.float() * torch.exp2(torch.arange(40, device="cuda") / 5 - 4)[:, None, None]).to(torch.bfloat16) for x in (k, v)]
    for t in range(40):
        b = Batch([t + 1], [t], [1], seed=0, max_pages=1, spare=3 - (t // 64 + 1), max_seq=64)
        want = _expected(b, kv8, k[t:t + 1], v[t:t + 1])
        dllm.dllm_kv8_write(_desc(2, 64), b.view.c, k[t:t + 1], v[t:t + 1], kv8.c)
        assert b.bits() == 0
        _assert_written(kv8, want)


def test_write_strided_rows():
    """Views of one projection output [M][(H + 2 kv) d], and heads that share one row of values."""
    b = Batch([80, 50], [10, 0], [33, 50])
    kv, d, H = 2, 128, 4
    qkv = torch.randn(b.M, (H + 2 * kv) * d, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, H * d:(H + kv) * d].view(b.M, kv, d), qkv[:, (H + kv) * d:].view(b.M, kv, d)
    for kk, vv in ((k, v), (k[:, :1].expand(-1, kv, -1), v), (k.flip(0).contiguous(), v[:1].expand(b.M, -1, -1))):
        kv8 = random_pools(b.num_pages, kv, d, 3)
        want = _expected(b, kv8, kk, vv)
        dllm.dllm_kv8_write(_desc(H, d), b.view.c, kk, vv, kv8.c)
        assert b.bits() == 0
        _assert_written(kv8, want)


@pytest.mark.parametrize("n,start,rows,kv,d", [w for w in WRITES if w[3] * w[4] % 128 == 0])
def test_write_from_the_bf16_pools(n, start, rows, kv, d):
    b = Batch(n, start, rows, seed=len(n))
    kv8 = random_pools(b.num_pages, kv, d, 3)
    cache = dllm.PagedCache(b.num_pages, kv, d)
    for t in (cache.k, cache.v):
        t.copy_(torch.randn(t.shape, device="cuda"))
    new = []
    for pool in (cache.k, cache.v):
        new.append(torch.stack([pool[b.table[i][p // PAGE], :, p % PAGE] for i in range(len(n))
                                for p in range(start[i], start[i] + rows[i])]))
    want = _expected(b, kv8, *new)
    dllm.dllm_kv8_write_pool(_desc(kv, d), b.view.c, cache.c, kv8.c)
    assert b.bits() == 0
    _assert_written(kv8, want)


def test_write_extreme_values():
    d = 128
    rows = torch.zeros(64, 1, d)
    rows[0:16, 0, :4] = torch.tensor([3e38, -3e38, 1e30, 1.0])   # beyond 448 * 2^60
    rows[16:32, 0, :4] = torch.tensor([float("inf"), float("nan"), 2.0, -float("inf")])
    rows[32:48, 0, :4] = torch.tensor([1e-38, -1e-38, 2e-40, 0.0])  # below the smallest scale
    b = Batch([64], [0], [64])
    kv8 = dllm.Kv8Cache(b.num_pages, 1, d)
    x = rows.cuda().to(torch.bfloat16)
    dllm.dllm_kv8_write(_desc(1, d), b.view.c, x, torch.zeros_like(x), kv8.c)
    assert b.bits() == dllm.DLLM_DEVERR_RANGE
    p = b.table[0][0]
    s = kv8.k_scale[p, 0].tolist()
    c = kv8.k.view(torch.uint8).view(torch.float8_e4m3fn).float()[p, 0].cpu()
    assert s[0] == 2.0 ** 60 and c[0, :4].tolist() == [448.0, -448.0, 448.0, 0.0]
    assert s[1] == 2.0 ** -7 and c[16, 2] == 256.0 and all(torch.isnan(c[16, i]) for i in (0, 1, 3)) and c[16, 4] == 0
    assert s[2] == 2.0 ** -60 and not c[32:48].any()
    assert s[3] == 2.0 ** -60 and not c[48:].any()
    assert kv8.v_scale[p, 0].tolist() == [2.0 ** -60] * 4


def test_write_scale_at_powers_of_two():
    """amax just at, below and above 448 times a power of two, over the whole range of exponents."""
    d = 64
    amax = torch.tensor([m * 2.0 ** e for e in range(-70, 68) for m in (446.0, 448.0, 450.0)])
    amax = amax[: len(amax) // 2 * 2]
    n = len(amax)
    rows = torch.zeros(n * G, 2, d)
    rows[::G, 0, 5] = amax
    rows[G - 1::G, 1, 0] = -amax
    b = Batch([n * G], [0], [n * G])
    kv8 = dllm.Kv8Cache(b.num_pages, 2, d)
    x = rows.cuda().to(torch.bfloat16)
    want = _expected(b, kv8, x, x)
    dllm.dllm_kv8_write(_desc(2, d), b.view.c, x, x, kv8.c)
    assert b.bits() == dllm.DLLM_DEVERR_RANGE
    _assert_written(kv8, want)


@pytest.mark.parametrize("change,bit", [
    (dict(table=[[99, 99], [2, 3]]), 2), (dict(table=[[-1, -1], [2, 3]]), 2), (dict(n=[1 << 20, 100]), 4),
    (dict(start=[-1, 90]), 4), (dict(start=[95, 90]), 4), (dict(rows=[9, 10]), 4), (dict(cub=[0, 10, 21]), 4)])
def test_write_skips_what_contradicts_the_bounds(change, bit):
    b = Batch([100, 100], [80, 90], [10, 10])
    b.t["table"].copy_(ints([[0, 1], [2, 3]]))
    b.table = [[0, 1], [2, 3]]
    kv8 = random_pools(6, 2, 64, 3)
    before = kv8.k.view(torch.uint8).clone()
    for k, v in change.items():
        b.t[k].copy_(ints(v))
    k, v = _rows(b.M, 2, 64, 4)
    dllm.dllm_kv8_write(_desc(2, 64), b.view.c, k, v, kv8.c)
    assert b.bits() == bit
    after = kv8.k.view(torch.uint8)
    assert torch.equal(after[[4, 5]], before[[4, 5]])
    if "rows" not in change and "cub" not in change:
        assert torch.equal(after[:2], before[:2])
        assert not torch.equal(after[3], before[3])  # the other sequence is written


# ------------------------------------------------------------------ the attention
def _ws(b, H, d, kv8):
    return dllm.workspace(dllm.dllm_kv8_attention_workspace_size(_desc(H, d), b.view.c, kv8.c))


def _q(M, H, d, seed, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(max(1, M), H, d, device="cuda", generator=g) * size).to(torch.bfloat16)


def _poison_tails(b, kv8):
    """Codes behind the end of each sequence's last page and the scales of whole groups there: not a number."""
    for i, n in enumerate(b.n):
        if n % PAGE:
            p = b.table[i][n // PAGE]
            for pool, scale in ((kv8.k, kv8.k_scale), (kv8.v, kv8.v_scale)):
                pool.view(torch.uint8)[p, :, n % PAGE:] = NAN_CODE
                scale[p, :, (n % PAGE + G - 1) // G:] = float("nan")


def _attend(b, q, kv8, ws=None, full=False, with_lse=True, fill=7.5):
    H, d = q.shape[1], q.shape[2]
    n = b.R if full else b.M
    o = torch.full((n, H, d), fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), fill, device="cuda") if with_lse else None
    ws = _ws(b, H, d, kv8) if ws is None else ws
    dllm.dllm_kv8_attention(_desc(H, d), b.view.c, q, kv8.c, o, lse, ws,
                            dllm.DLLM_ROWS_FULL if full else dllm.DLLM_ROWS_BLOCK)
    return o, lse


ATTEND = [
    # lengths, block starts, block lengths, heads, kv heads, d
    ([1], [0], [1], 1, 1, 128),
    ([1], [0], [1], 2, 2, 64),
    ([63, 64, 65, 127, 128, 129], [0, 10, 64, 100, 96, 128], [1, 3, 1, 27, 32, 1], 2, 1, 128),
    ([63, 64, 65, 127, 128, 129], [0, 10, 64, 100, 96, 128], [1, 3, 1, 27, 32, 1], 4, 2, 64),
    ([320], [32], [32], 4, 4, 64),
    ([0, 40, 0, 200, 0], [0, 39, 0, 0, 0], [0, 1, 0, 64, 0], 3, 3, 128),
    ([100, 0, 50], [5, 0, 0], [0, 0, 50], 4, 1, 128),             # a sequence without rows beside one with
    ([500, 333], [100, 200], [16, 33], 5, 1, 128),                # 5 query heads to a key head: 80 and 165 rows
    ([200, 100], [0, 0], [200, 100], 6, 2, 64),                   # whole prompts as blocks
    ([700], [37], [1], 32, 1, 128),
    ([1000, 3], [900, 2], [9, 1], 56, 8, 128),                    # 7 to a head
    ([2500, 64, 1], [2400, 0, 0], [64, 64, 1], 2, 2, 128),
    ([5000, 4097, 31], [4990, 0, 30], [1, 1, 1], 8, 2, 128),
    ([5000, 4097, 31], [4990, 0, 30], [4, 7, 1], 8, 2, 64),
]


@pytest.mark.parametrize("n,start,rows,H,kv,d", ATTEND)
def test_attention(n, start, rows, H, kv, d):
    if H * d % 128:
        H, kv = 2 * H, 2 * kv
    b = Batch(n, start, rows, seed=sum(n), cap_rows=sum(rows) + 2, cap_seq=sum(n) + 2, max_block=max(rows) + 2,
              max_seq=max(n) + 2, max_pages=max(n) // 64 + 1)
    kv8 = random_pools(b.num_pages, kv, d, sum(n))
    _poison_tails(b, kv8)
    q = _q(b.M, H, d, 9)
    ref = attention(b, q, kv8)
    o, lse = _attend(b, q, kv8)
    assert b.bits() == 0
    assert_attention(b, q, kv8, o, lse, ref=ref)
    M = sum(rows)
    assert (o[M:] == 7.5).all() and (lse[M:] == 7.5).all()  # rows behind the last sequence are left
    # the full layout: the same bits at the rows of the whole sequences, and no other row
    of, lf = _attend(b, q, kv8, full=True)
    at = torch.cat([torch.arange(s, s + r) + c for s, r, c in zip(start, rows, np.cumsum([0] + n[:-1]).tolist())]).cuda().long()
    assert torch.equal(of[at], o[:M]) and torch.equal(lf[at], lse[:M])
    rest = torch.ones(b.R, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (of[rest] == 7.5).all() and (lf[rest] == 7.5).all()
    assert torch.equal(_attend(b, q, kv8, with_lse=False)[0], o)
    assert b.bits() == 0


@pytest.mark.parametrize("seed", range(6))
def test_attention_random_shapes(seed):
    r = random.Random(100 + seed)
    d = r.choice([64, 128])
    kv = r.choice([1, 2, 3, 4]) * (128 // d)
    H = kv * r.choice([1, 2, 3, 4, 8])
    batch = r.randint(1, 40)
    n = [r.choice([r.randint(1, 300), r.randint(1, 3000)]) for _ in range(batch)]
    rows = [r.randint(1, min(x, 70)) for x in n]
    start = [r.randint(0, x - k) for x, k in zip(n, rows)]
    b = Batch(n, start, rows, seed=seed)
    kv8 = random_pools(b.num_pages, kv, d, seed, spread=1.0)
    _poison_tails(b, kv8)
    q = _q(b.M, H, d, seed)
    o, lse = _attend(b, q, kv8)
    assert b.bits() == 0
    assert_attention(b, q, kv8, o, lse)


@pytest.mark.parametrize("H,kv,rows", [(2, 2, 20), (8, 1, 1), (4, 2, 40)])
@pytest.mark.parametrize("how", ["large scores", "rising scores", "one key takes nearly all", "scales far apart", "a zero group",
                                 "small values", "large values"])
def test_attention_hard_values(how, H, kv, rows):
    n, d = 1500, 128
    b = Batch([n, 700], [n - rows, 0], [rows, rows], seed=3)
    kv8 = random_pools(b.num_pages, kv, d, 5)
    q = _q(b.M, H, d, 6, size=20.0 if how == "large scores" else 1.0)
    if how == "rising scores":  # every group's keys larger than the last: the reference moves again and again
        for i, m in enumerate(b.n):
            for p in range((m + 63) // 64):
                kv8.k_scale[b.table[i][p]] *= 2.0 ** (p // 4 - 2)
    elif how == "one key takes nearly all":  # and a long tail that together weighs as much
        kv8.k_scale.mul_(0.01)
        page = b.table[0][0]
        kv8.k_scale[page, :, 0] = 1.0
        kv8.k.view(torch.uint8)[page, :, 0:16] = 0
        kv8.k.view(torch.uint8)[page, :, 0] = (q[0, 0].float() * 7.3 / q[0, 0].float().pow(2).sum() * d ** 0.5).to(
            torch.float8_e4m3fn).view(torch.uint8)
    elif how == "scales far apart":
        g = torch.Generator("cuda").manual_seed(1)
        kv8.v_scale.mul_(torch.exp2(torch.randint(-20, 21, kv8.v_scale.shape, device="cuda", generator=g).float()))
        kv8.v_scale[b.table[0][0]] = 2.0 ** -60
    elif how == "a zero group":
        kv8.v.view(torch.uint8)[b.table[0][1]] = 0
        kv8.v_scale[b.table[0][1]] = 2.0 ** -60
        kv8.k.view(torch.uint8)[b.table[0][2]] = 0
        kv8.k_scale[b.table[0][2]] = 2.0 ** -60
    elif how == "small values":
        kv8.v_scale.mul_(2.0 ** -40)
    elif how == "large values":
        kv8.v_scale.mul_(2.0 ** 60)
    o, lse = _attend(b, q, kv8)
    assert b.bits() == 0
    assert_attention(b, q, kv8, o, lse)


def test_attention_scales_that_are_no_powers_of_two():
    b = Batch([400, 77], [300, 0], [32, 32], seed=3)
    kv8 = random_pools(b.num_pages, 2, 128, 5)
    kv8.k_scale.mul_(1.0 + torch.rand(kv8.k_scale.shape, device="cuda"))
    kv8.v_scale.mul_(1.0 + torch.rand(kv8.v_scale.shape, device="cuda"))
    q = _q(b.M, 4, 128, 6)
    o, lse = _attend(b, q, kv8)
    assert_attention(b, q, kv8, o, lse)


def test_attention_scale_and_strided_queries():
    b = Batch([300, 100], [100, 0], [32, 17], seed=3)
    kv8 = random_pools(b.num_pages, 2, 128, 5)
    wide = _q(b.M, 8, 128, 6)
    q = wide[:, 2:6]
    o = torch.zeros(b.M, 4, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(b.M, 4, device="cuda")
    desc = dllm.layer_desc(512, 4, 128, 1e4, softmax_scale=0.03125)
    dllm.dllm_kv8_attention(desc, b.view.c, q, kv8.c, o, lse, _ws(b, 4, 128, kv8))
    assert_attention(b, q, kv8, o, lse, scale=0.03125)


@pytest.mark.parametrize("batch,longest,H,kv,d", [(129, 300, 2, 1, 128), (300, 700, 4, 4, 64), (700, 200, 16, 2, 64), (1500, 400, 2, 2, 64)])
def test_attention_large_batches(batch, longest, H, kv, d):
    """More sequences than one warp sums up, places without a request among them."""
    r = random.Random(batch)
    n = [r.choice([0, 1, r.randint(1, longest), r.randint(1, longest)]) for _ in range(batch)]
    rows = [min(x, r.choice([0, 1, 1, 4])) for x in n]
    start = [r.randint(0, x - k) for x, k in zip(n, rows)]
    b = Batch(n, start, rows, seed=batch, max_block=4, max_seq=longest)
    kv8 = random_pools(b.num_pages, kv, d, batch)
    _poison_tails(b, kv8)
    q = _q(b.M, H, d, 9)
    o, lse = _attend(b, q, kv8)
    assert b.bits() == 0
    assert_attention(b, q, kv8, o, lse)


@pytest.mark.parametrize("longest", [512, 513])
def test_attention_with_and_without_cuts(longest):
    """Sequences of up to 512 tokens are attended to whole, longer ones in pieces: the same inputs under either bound."""
    n = [512, 300, 1, 129, 64, 512]
    b = Batch(n, [480, 0, 0, 100, 0, 0], [32, 32, 1, 29, 1, 8], seed=1, max_seq=longest, max_pages=9)
    kv8 = random_pools(b.num_pages, 4, 128, 5)
    _poison_tails(b, kv8)
    q = _q(b.M, 8, 128, 6)
    o, lse = _attend(b, q, kv8)
    assert b.bits() == 0
    assert_attention(b, q, kv8, o, lse)


def test_attention_one_head_over_the_whole_gpu():
    """A single unit: every CTA has a piece of it, and the join more than it takes at a time."""
    b = Batch([60000], [59999], [1], seed=1)
    kv8 = random_pools(b.num_pages, 1, 128, 5, spread=1.0)
    q = _q(1, 5, 128, 6)
    o, lse = _attend(b, q, kv8)
    assert b.bits() == 0
    assert_attention(b, q, kv8, o, lse)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [200, 3000])
def test_attention_not_a_number_in_a_query_stays_in_its_row(value, n):
    b = Batch([n, 77], [100, 0], [8, 8], seed=3)
    kv8 = random_pools(b.num_pages, 2, 128, 5)
    q = _q(b.M, 4, 128, 6)
    ref = attention(b, q, kv8)
    bad = q.clone()
    bad[3, 1, 17] = value
    o, lse = _attend(b, bad, kv8)
    assert torch.isnan(o[3, 1]).all() and torch.isnan(lse[3, 1])
    o[3, 1], lse[3, 1] = ref[0][3, 1].to(torch.bfloat16), ref[1][3, 1].float()
    assert_attention(b, q, kv8, o, lse, ref=ref)


def test_attention_zero_and_tiny_queries():
    """A query of zeros weighs all keys alike; one far smaller than the others of its unit still has its own scores."""
    b = Batch([300], [100], [4], seed=3)
    kv8 = random_pools(b.num_pages, 1, 128, 5)
    q = _q(4, 2, 128, 6)
    q[0] = 0
    q[1] *= 2.0 ** -9
    o, lse = _attend(b, q, kv8)
    assert_attention(b, q, kv8, o, lse)
    assert (lse[0] - np.log(300)).abs().max() < 1e-5
    o, lse = _attend(b, torch.zeros_like(q), kv8)
    assert_attention(b, torch.zeros_like(q), kv8, o, lse)


def test_attention_not_a_number_stays_in_its_head():
    """A not-a-number code among the attended keys or values makes its (sequence, key head) not a number, and no other."""
    b = Batch([200, 300], [100, 0], [8, 8], seed=3)
    for pool in ("k", "v"):
        kv8 = random_pools(b.num_pages, 2, 128, 5)
        q = _q(b.M, 4, 128, 6)
        want, wl = _attend(b, q, kv8)
        getattr(kv8, pool).view(torch.uint8)[b.table[0][1], 0, 7, 3] = NAN_CODE
        o, lse = _attend(b, q, kv8)
        if pool == "k":
            assert torch.isnan(o[:8, :2]).all() and torch.isnan(lse[:8, :2]).all()
        else:
            assert torch.isnan(o[:8, :2, 3]).all() and torch.equal(lse, wl)
        assert torch.equal(o[:8, 2:], want[:8, 2:]) and torch.equal(o[8:], want[8:])


def test_attention_repeats_bit_for_bit_whatever_the_workspace_holds():
    b = Batch([40000, 3, 700], [39990, 0, 5], [4, 3, 64], seed=3)
    kv8 = random_pools(b.num_pages, 2, 128, 5)
    q = _q(b.M, 8, 128, 6)
    ws = _ws(b, 8, 128, kv8)
    first = _attend(b, q, kv8, ws)
    for _ in range(5):
        again = _attend(b, q, kv8, ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
        ws.fill_(0xFF)
    assert_attention(b, q, kv8, *first)
    # the workspace serves another shape next
    c = Batch([900, 12000], [0, 11000], [1, 1], seed=4)
    kv8c = random_pools(c.num_pages, 2, 128, 6)
    qc = _q(c.M, 4, 128, 7)
    assert_attention(c, qc, kv8c, *_attend(c, qc, kv8c, ws))


def test_attention_page_order_does_not_matter():
    outs = []
    for seed in (1, 2):
        b = Batch([3000, 200], [1000, 0], [32, 32], seed=seed)
        kv8 = random_pools(b.num_pages, 2, 64, 5)
        canon = dllm.Kv8Cache(b.num_pages, 2, 64)
        order = [p for t in b.table for p in t if p >= 0]
        for dst, src in ((canon.k.view(torch.uint8), kv8.k.view(torch.uint8)), (canon.v.view(torch.uint8), kv8.v.view(torch.uint8)),
                         (canon.k_scale, kv8.k_scale), (canon.v_scale, kv8.v_scale)):
            dst[order] = src[:len(order)]
        outs.append(_attend(b, _q(b.M, 4, 64, 6), canon))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("change,bit", [
    (dict(table=[[99, 99], [2, 3]]), 2), (dict(table=[[-1, -1], [2, 3]]), 2), (dict(n=[1 << 20, 100]), 4), (dict(n=[-5, 100]), 4),
    (dict(start=[-1, 90]), 4), (dict(start=[95, 90]), 4), (dict(rows=[-9, 10]), 4), (dict(rows=[11, 10]), 4),
    (dict(cub=[15, 10, 20]), 4), (dict(cub=[-1, 10, 20]), 4)])
def test_attention_refuses_what_contradicts_the_bounds(change, bit):
    b = Batch([100, 100], [80, 90], [10, 10])
    b.t["table"].copy_(ints([[0, 1], [2, 3]]))
    b.table = [[0, 1], [2, 3]]
    kv8 = random_pools(6, 2, 64, 3)
    q = _q(b.M, 4, 64, 1)
    for k, v in change.items():
        b.t[k].copy_(ints(v))
    o, lse = _attend(b, q, kv8)
    assert b.bits() == bit
    o64 = attention(b, q, kv8)[0]
    assert (o[10:].double() - o64[10:]).abs().max() < 0.02  # the other sequence is attended to


def test_offsets_beyond_32_bits():
    """Pools of more than 4 GB, the sequences in their last pages."""
    kv, d, P = 32, 128, 17000
    b = Batch([300, 70], [200, 0], [32, 32], seed=1, first_page=P - 9)
    assert b.num_pages <= P and P * kv * PAGE * d > 1 << 32
    kv8 = dllm.Kv8Cache(P, kv, d)
    k, v = _rows(370, kv, d, 2)
    whole = Batch([300, 70], [0, 0], [300, 70], seed=1, first_page=P - 9)
    dllm.dllm_kv8_write(_desc(kv, d), whole.view.c, k, v, kv8.c)
    assert not kv8.k.view(torch.uint8)[:P - 9].any()
    q = _q(b.M, kv, d, 3)
    o, lse = _attend(b, q, kv8)
    assert b.bits() == 0 and whole.bits() == 0
    assert_attention(b, q, kv8, o, lse)


def test_two_streams_at_once():
    bs = [Batch([3000, 500], [100, 0], [32, 32], seed=s) for s in (1, 2)]
    kv8 = [random_pools(b.num_pages, 2, 128, 7 + i) for i, b in enumerate(bs)]
    qs = [_q(b.M, 4, 128, i) for i, b in enumerate(bs)]
    want = [_attend(b, q, k) for b, q, k in zip(bs, qs, kv8)]
    ws = [_ws(b, 4, 128, k) for b, k in zip(bs, kv8)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(_attend(bs[i], qs[i], kv8[i], ws[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


# ------------------------------------------------------------------ together
def test_a_captured_serving_loop():
    """Plan, write and attention captured once and replayed while requests grow, end and come: the lengths change between
    replays, the addresses do not.  Each step against the plain forms."""
    kv, H, d, batch, width, P = 2, 8, 128, 6, 16, 40
    r = random.Random(3)
    dev = dict(table=ints([[0] * 8] * batch), n=ints([0] * batch), start=ints([0] * batch), rows=ints([0] * batch),
               cub=ints([0] * (batch + 1)), cus=ints([0] * (batch + 1)), held=ints([0] * batch), held_out=ints([0] * batch),
               err=ints([0]))
    ring = dllm.PageRing.full(P)
    cap = batch * width
    view = dllm.BatchView(dev["table"], dev["n"], dev["start"], dev["rows"], dev["cub"], dev["cus"], cap, batch * 512, width, 512,
                          dev["err"])
    kv8 = dllm.Kv8Cache(P, kv, d)
    desc = _desc(H, d)
    ws = dllm.workspace(dllm.dllm_kv8_attention_workspace_size(desc, view.c, kv8.c))
    q, o = _q(cap, H, d, 1), torch.zeros(cap, H, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(cap, H, device="cuda")
    k, v = _rows(cap, kv, d, 2)

    def step():
        dllm.dllm_batch_plan(view.c, dev["held"], dev["held_out"], dev["table"], dev["cub"], dev["cus"], ring.c)
        dllm.dllm_kv8_write(desc, view.c, k, v, kv8.c)
        dllm.dllm_kv8_attention(desc, view.c, q, kv8.c, o, lse, ws)
        dev["held"].copy_(dev["held_out"])
        ring.state.copy_(ring.state_out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # nothing planned yet: an empty batch
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    n = [0] * batch
    for i in range(25):
        new = [r.choice([0, 1, r.randint(1, width)]) for _ in range(batch)]
        n = [0 if r.random() < 0.1 else x for x in n]
        new = [min(c, 400 - x) for c, x in zip(new, n)]
        start, n = n, [x + c for x, c in zip(n, new)]
        for key, val in (("n", n), ("start", start), ("rows", new)):
            dev[key].copy_(ints(val))
        k2, v2 = _rows(cap, kv, d, 50 + i, size=1.0 + i)
        k.copy_(k2)
        v.copy_(v2)
        o.fill_(3.0)
        before = [t.clone() for t in (kv8.k.view(torch.uint8), kv8.v.view(torch.uint8), kv8.k_scale, kv8.v_scale)]
        graph.replay()
        torch.cuda.synchronize()
        assert dev["err"].item() == 0
        b = Batch([1], [0], [1])
        b.n, b.start, b.rows, b.table, b.M = n, start, new, dev["table"].tolist(), cap
        old = dllm.Kv8Cache.of(before[0].view(torch.float8_e4m3fn), before[1].view(torch.float8_e4m3fn), *before[2:])
        _assert_written(kv8, _expected(b, old, k, v))
        assert_attention(b, q, kv8, o, lse)
        assert (o[sum(new):] == 3.0).all()


def test_beside_the_bf16_cache():
    """A block boundary and an inner step of the tiny workload: the 8-bit cache written out of the bf16 pools and attended
    to beside dllm_block_attention, in the layout of its outputs.  The two differ by what e4m3 rounds away: at most
    2^-4 of each key and value."""
    cfg = make_config("tiny")
    wl = Workload(cfg)
    st = LayerStep(cfg, blocks=[2], weights=wl.weights(0))
    st.boundary(full_rows_of(wl, 0, 0, [2]).cuda())
    kv8 = dllm.Kv8Cache(st.cache.num_pages, cfg.n_heads, cfg.head_dim)
    n = cfg.seq_len(0)
    whole = st.batch.with_blocks([0], [n])
    dllm.dllm_kv8_write_pool(st.desc, whole.c, st.cache.c, kv8.c)
    x = block_rows_of(wl, 0, 1, [2]).cuda()
    st.step(x)
    dllm.dllm_kv8_write_pool(st.desc, st.batch.c, st.cache.c, kv8.c)
    o = torch.zeros_like(st.o_full)
    ws = dllm.workspace(dllm.dllm_kv8_attention_workspace_size(st.desc, st.batch.c, kv8.c))
    dllm.dllm_kv8_attention(st.desc, st.batch.c, st.q_block.view(-1, cfg.n_heads, cfg.head_dim), kv8.c, o, None, ws,
                            dllm.DLLM_ROWS_FULL)
    torch.cuda.synchronize()
    assert st.batch.error_bits() == 0
    s, k = cfg.block_start(0, 2), cfg.block[0]
    b = Batch([n], [s], [k])
    b.table = st.batch.host["block_table"].tolist()
    rows = o.view(-1, cfg.n_heads, cfg.head_dim)[s:s + k]
    assert_attention(b, st.q_block.view(-1, cfg.n_heads, cfg.head_dim), kv8, rows, None)
    pages = torch.tensor(b.table[0][:(n + 63) // 64], device="cuda")
    for pool, codes, scale in ((st.cache.k, kv8.k, kv8.k_scale), (st.cache.v, kv8.v, kv8.v_scale)):
        a, c = (t.transpose(0, 1).reshape(cfg.n_heads, -1, cfg.head_dim)[:, :n] for t in
                (pool[pages].double(), values(codes[pages], scale[pages])))
        group = a.abs().amax(-1, keepdim=True)
        assert ((a - c).abs() <= 2.0 ** -4 * a.abs() + 2.0 ** -10 * group.amax(1, keepdim=True) / 224).all()
    full = st.o_full.view(-1, cfg.n_heads, cfg.head_dim)[s:s + k].double()
    assert (rows.double() - full).norm() <= 2.0 ** -3 * full.norm()
