"""The 8-bit attention where the rows of a unit of work differ: each row keeps its own precision."""
import math

import pytest
import torch

from block_wise_kv_gb300 import dllm
from kv8_util import Batch, attention, random_pools

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_wise_kv_gb300 import build

    build.build()
    dllm.load()
    torch.cuda.init()


def _attend(b, q, kv8):
    H, d = q.shape[1], q.shape[2]
    desc = dllm.layer_desc(max(64, H * d), H, d, 1e4)
    o = torch.full((b.M, H, d), 7.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.M, H), 7.5, device="cuda")
    ws = dllm.workspace(dllm.dllm_kv8_attention_workspace_size(desc, b.view.c, kv8.c))
    dllm.dllm_kv8_attention(desc, b.view.c, q, kv8.c, o, lse, ws)
    assert b.bits() == 0
    return o, lse


def _assert_rows(b, q, kv8, o, lse, of=None):
    """Bounds row by row (`of`: those that are looked at, [M][H]).  A row's q is held in two e4m3 parts of q 2^-e, the
    row's largest in (224, 448]: a value is off by half of e4m3's smallest step at most, 2^-10, that is 2^-17.8 of the
    row's largest.  A score is a sum of eight 32-bit steps at most (2^-23 of what is summed each, 2^-20 in all) and is
    scaled and shifted in 32 bits (2^-22).  Together less than e = 2^-17 max|q| sum|k| of the row, which moves a weight
    by a factor of exp(2 e) at most.  The output is rounded to bf16 (2^-8), the weights to 11 bits (2^-11, as much again for the
    exponential and the sums) and to an absolute 2^-27 of the row's largest weight x value scale for each code."""
    o64, lse64, a64, reach, small = attention(b, q, kv8)
    e = 2.0 ** -17 * q.double().abs().amax(-1) * reach
    tol = 2.0 ** -8 * o64.abs() + (2.0 ** -10 + torch.expm1(2 * e))[..., None] * a64 + 2.0 ** -27 * small
    bad = ~((o.double() - o64).abs() <= tol)
    ltol = e + 2.0 ** -20 * (1 + lse64.abs())
    lbad = ~((lse.double() - lse64).abs() <= ltol)
    if of is not None:
        bad, lbad = bad & of[..., None], lbad & of
    assert not lbad.any(), (int(lbad.sum()), lbad.nonzero()[0].tolist(), float(lse[lbad][0]), float(lse64[lbad][0]))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float(o[bad][0]), float(o64[bad][0]))


SHAPES = [(8, 1, 1, 64), (8, 1, 2, 128), (2, 2, 20, 128), (4, 4, 30, 64), (4, 2, 40, 128), (4, 2, 40, 64)]  # H, kv, rows, d


def _setup(H, kv, rows, d, seed=0):
    b = Batch([700, 330], [700 - rows, 5], [rows, rows], seed=3)
    kv8 = random_pools(b.num_pages, kv, d, 5 + seed)
    g = torch.Generator("cuda").manual_seed(6 + seed)
    return b, kv8, torch.randn(b.M, H, d, device="cuda", generator=g)


@pytest.mark.parametrize("H,kv,rows,d", SHAPES)
@pytest.mark.parametrize("shift", [6, 12, 20, 40])
def test_a_row_far_smaller_than_its_neighbours_keeps_its_scores(H, kv, rows, d, shift):
    """Every second (row, head) is 2^-shift of the others, and the keys are 2^shift as large: the small rows' scores are
    ordinary ones."""
    b, kv8, q = _setup(H, kv, rows, d)
    odd = (torch.arange(H, device="cuda")[None] + torch.arange(b.M, device="cuda")[:, None]) % 2 == 1
    q[odd] *= 2.0 ** -shift
    kv8.k_scale.mul_(2.0 ** shift)
    q = q.to(torch.bfloat16)
    o, lse = _attend(b, q, kv8)
    _assert_rows(b, q, kv8, o, lse, odd)


@pytest.mark.parametrize("H,kv,rows,d", SHAPES)
@pytest.mark.parametrize("value", [1e4, 1e30, -3e38])
def test_one_large_value_leaves_the_other_rows_as_they_are(H, kv, rows, d, value):
    b, kv8, q = _setup(H, kv, rows, d, 1)
    q = q.to(torch.bfloat16)
    q[rows // 2, 1, 17] = value
    o, lse = _attend(b, q, kv8)
    others = torch.ones(b.M, H, dtype=torch.bool, device="cuda")
    others[rows // 2, 1] = False
    _assert_rows(b, q, kv8, o, lse, others)
    # the same bits as without it
    q[rows // 2, 1, 17] = 1.0
    again = _attend(b, q, kv8)
    assert torch.equal(again[0][others], o[others]) and torch.equal(again[1][others], lse[others])


@pytest.mark.parametrize("H,kv,rows,d", SHAPES)
def test_rows_of_all_magnitudes(H, kv, rows, d):
    """Rows from 2^-100 to 2^12 of ordinary ones: the larger the sharper, the smallest weigh all keys alike."""
    b, kv8, q = _setup(H, kv, rows, d, 2)
    n = b.M * H
    q = (q.view(n, d) * torch.exp2(torch.linspace(-100, 12, n, device="cuda").round())[:, None]).view(b.M, H, d).to(torch.bfloat16)
    o, lse = _attend(b, q, kv8)
    _assert_rows(b, q, kv8, o, lse)


@pytest.mark.parametrize("H,kv,rows,d", SHAPES)
def test_the_largest_scores(H, kv, rows, d):
    """Scores of up to 2^25 in magnitude: each row takes the value of its largest key (exact powers of two throughout, so
    that nothing but that decides), rising tile after tile so that the reference moves too."""
    b, kv8, _ = _setup(H, kv, rows, d, 3)
    q = torch.zeros(b.M, H, d, device="cuda", dtype=torch.bfloat16)
    q[:, :, 3] = 2.0 ** 14
    kv8.k.view(torch.uint8).zero_()
    kv8.k_scale.fill_(1.0)
    tops = []
    for i, n in enumerate(b.n):
        for p in range(0, n, 64):
            page = b.table[i][p // 64]
            kv8.k.view(torch.uint8)[page, :, min(63, n - p - 1), 3] = 0x38  # 1.0
            kv8.k_scale[page, :, min(63, n - p - 1) // 16] = 2.0 ** (4 + p // 64)
        tops.append((b.table[i][(n - 1) // 64], (n - 1) % 64))
    assert 2.0 ** 14 * 2.0 ** (4 + 699 // 64) / math.sqrt(d) <= 2.0 ** 25
    o, lse = _attend(b, q, kv8)
    at = 0
    for (page, slot), r in zip(tops, b.rows):
        v = kv8.v[page, :, slot].float() * kv8.v_scale[page, :, slot // 16, None]
        want = v.to(torch.bfloat16).repeat_interleave(H // kv, 0)
        # the weight is 1, held in 11 bits and summed in 32: at most 2^-11 beside the bf16 step
        assert ((o[at:at + r].float() - want.float()).abs() <= (2.0 ** -7 + 2.0 ** -11) * want.float().abs()).all()
        score = 2.0 ** 14 * 2.0 ** (4 + (b.n[0 if at == 0 else 1] - 1) // 64) * d ** -0.5
        assert ((lse[at:at + r] - score).abs() <= 2.0 ** -21 * score).all()
        at += r
