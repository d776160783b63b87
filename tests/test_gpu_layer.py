"""A layer's products, the norm and rotation of its heads, and token scores on the GPU, each against a plain 64-bit
implementation (tests/layer_util.py), and a run of them together with the 8-bit cache."""
import math

import pytest
import torch

import layer_util as lu
from block_wise_kv_gb300 import dllm
from kv8_util import Batch, assert_attention, ints

pytestmark = pytest.mark.gpu
ACT = {"none": dllm.DLLM_ACT_NONE, "silu": dllm.DLLM_ACT_SILU, "gelu": dllm.DLLM_ACT_GELU,
       "gelu_tanh": dllm.DLLM_ACT_GELU_TANH}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_wise_kv_gb300 import build

    build.build()
    dllm.load()
    torch.cuda.init()


# ------------------------------------------------------------------ products with a weight
class Linear:
    def __init__(self, m, k, n, name="none", gated=False, norm=False, bias=False, residual=False, pad=0, seed=0, size=1.0):
        wide = 2 * n if gated else n
        self.m, self.n, self.name, self.gated = m, n, name, gated
        self.x = lu.randn((m, k + 8 * pad), seed, size)[:, :k]
        self.w = lu.randn((wide, k), seed + 1, 1.0 / math.sqrt(k))
        self.gain = (1 + lu.randn((k,), seed + 2, 0.2).float()).bfloat16() if norm else None
        self.bias = lu.randn((wide,), seed + 3) if bias else None
        self.residual = lu.randn((m, n + pad), seed + 4)[:, :n] if residual else None
        self.whole = torch.full((m, n + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        self.y = self.whole[:, :n]
        self.desc = dllm.linear_desc(k, n, ACT[name], gated, 1e-5)
        self.ws = dllm.workspace(dllm.dllm_linear_workspace_size(self.desc, m, norm)) if norm else None
        self.error = ints([0])

    def call(self, **kw):
        dllm.dllm_linear(self.desc, self.x, self.w, self.y, **{**dict(
            rms_gain=self.gain, bias=self.bias, residual=self.residual, ws=self.ws, error=self.error), **kw})

    def check(self, y=None, residual=None):
        y = self.y if y is None else y
        want, off = lu.linear(self.x, self.w, self.gain, self.bias, self.residual if residual is None else residual,
                              self.name, self.gated)
        err = (y.double() - want).abs()
        assert (err <= off).all(), (err.max().item(), (err / off).max().item())
        assert self.error.item() == 0
        assert (self.whole[:, self.n:] == 7.0).all()


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 100, 128, 255, 256, 257, 513])
@pytest.mark.parametrize("k,n", [(64, 128), (256, 768), (1000, 130)])
def test_linear_rows(m, k, n):
    c = Linear(m, k, n, residual=m % 2 == 0, bias=m % 3 == 0, seed=m)
    c.call()
    c.check()


@pytest.mark.parametrize("k", [8, 16, 56, 72, 120, 136, 520, 4096, 12288])
@pytest.mark.parametrize("n,m", [(1, 3), (127, 1), (129, 40), (200, 300)])
def test_linear_sizes(k, n, m):
    c = Linear(m, k, n, bias=True, residual=True, pad=1, seed=k + n)
    c.call()
    c.check()


@pytest.mark.parametrize("name", lu.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n", [(1, 64), (37, 100), (300, 333), (700, 1024)])
def test_linear_epilogues(name, gated, m, n):
    for bias, residual, norm in ((False, False, False), (True, True, False), (False, True, True), (True, False, True)):
        c = Linear(m, 192, n, name, gated, norm, bias, residual, pad=3 if residual else 0, seed=n, size=2.0)
        c.call()
        c.check()


def test_linear_large_arguments_of_the_activations():
    for name in lu.ACTS:
        c = Linear(70, 64, 96, name, seed=5, size=60.0)
        c.call()
        c.check()


@pytest.mark.parametrize("m,k,n,gated", [(512, 1024, 3000, False), (2048, 512, 1500, True), (5000, 264, 520, False)])
def test_linear_many_rows(m, k, n, gated):
    c = Linear(m, k, n, "silu" if gated else "none", gated, norm=gated, residual=not gated, seed=m)
    c.call()
    c.check()


@pytest.mark.parametrize("m,k", [(33, 16), (900, 1016), (1500, 1032), (1100, 2984), (257, 4096), (600, 4104), (40, 12288),
                                 (3, 16392)])
@pytest.mark.parametrize("size", [1.0, 1e-4, 3e4])
def test_linear_norm_of_rows_of_any_length(m, k, size):
    c = Linear(m, k, 72, norm=True, pad=1, seed=k, size=size)
    c.call()
    c.check()


@pytest.mark.parametrize("k", [8, 248, 264, 2048, 2056, 4096, 4104, 8192, 8200, 12344, 16384, 16392])
@pytest.mark.parametrize("n,gated", [(1, False), (1, True), (37, True), (305, False), (1219, False)])
@pytest.mark.parametrize("m", [1, 2])
def test_linear_few_rows(m, k, n, gated):
    for bias, residual, norm in ((False, False, False), (True, True, True)):
        c = Linear(m, k, n, "silu" if gated else "none", gated, norm, bias, residual, pad=m - 1, seed=k + n)
        c.call()
        c.check()


@pytest.mark.parametrize("m,k,n,gated", [(1, 8, 60000, True), (1, 72, 200000, False), (2, 16, 100003, False),
                                         (2, 8, 40001, True)])
def test_linear_few_rows_of_many_columns(m, k, n, gated):
    c = Linear(m, k, n, "gelu" if gated else "none", gated, bias=True, residual=True, pad=3, seed=n)
    c.call()
    c.check()


def test_linear_values_that_are_not_finite_stay_in_their_row():
    c = Linear(40, 128, 200, seed=3)
    c.x[7, 5] = math.nan
    c.x[9, 9] = math.inf
    c.call()
    assert torch.isnan(c.y[7]).all() and not torch.isfinite(c.y[9]).any()
    keep = [i for i in range(40) if i not in (7, 9)]
    want, off = lu.linear(c.x[keep], c.w)
    assert ((c.y[keep].double() - want).abs() <= off).all()


@pytest.mark.parametrize("m,n,pad", [(1, 640, 0), (96, 640, 8), (600, 640, 0), (600, 641, 2)])
def test_linear_adds_to_the_residual_in_place(m, n, pad):
    c = Linear(m, 256, n, residual=True, pad=pad, seed=m)
    before = c.residual.clone()
    whole = torch.full_like(c.whole, 7.0)
    y = whole[:, :n]
    y.copy_(before)
    dllm.dllm_linear(c.desc, c.x, c.w, y, residual=y)
    c.check(y, before)
    assert (whole[:, n:] == 7.0).all()


def test_linear_out_of_and_into_columns_of_one_buffer():
    wide = lu.randn((50, 64 + 96 + 40), 1)
    x, y = wide[:, :64], wide[:, 64:160]
    w = lu.randn((96, 64), 2, 0.1)
    want, off = lu.linear(x, w)
    kept = wide[:, 160:].clone()
    dllm.dllm_linear(dllm.linear_desc(64, 96), x, w, y)
    assert ((y.double() - want).abs() <= off).all() and torch.equal(wide[:, 160:], kept)


def test_linear_gives_the_same_bits_again_and_rows_do_not_see_each_other():
    for m, k, n in ((3, 4096, 512), (64, 4096, 512), (300, 1024, 700), (1024, 2048, 512)):
        c = Linear(m, k, n, "silu", norm=True, seed=m)
        c.call()
        first = c.y.clone()
        c.x[m // 2 + 1:] = 0
        c.call()
        assert torch.equal(c.y[:m // 2 + 1], first[:m // 2 + 1])


def test_linear_on_two_streams_and_captured():
    cs = [Linear(48, 1024, 640, norm=True, residual=True, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                c.call()
    torch.cuda.synchronize()
    for c in cs:
        c.check()
    c = cs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for seed in (11, 12):
        c.x.copy_(lu.randn(c.x.shape, seed))
        c.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check()


def test_linear_sees_what_the_kernel_before_it_wrote():
    """Weights, rows and residual written by the kernel directly in front, and rows read by the one behind, over and over."""
    c = Linear(64, 2048, 1024, residual=True, seed=1)
    ws = [c.w.clone(), lu.randn(c.w.shape, 9, 0.02)]
    xs = [c.x.clone(), lu.randn(c.x.shape, 8)]
    want = []
    for w, x in zip(ws, xs):
        c.w.copy_(w)
        c.x.copy_(x)
        torch.cuda.synchronize()
        c.call()
        want.append(c.y.clone())
    for i in range(40):
        c.x.copy_(xs[i % 2])
        c.w.copy_(ws[i % 2])
        c.call()
        got = c.y.clone()
        assert torch.equal(got, want[i % 2])


# ------------------------------------------------------------------ head norms and rotation
def _heads(m, h, d, seed, layout):
    if layout == "rows":
        return lu.randn((m, h, d), seed)
    if layout == "wide":  # heads out of a wider row
        return lu.randn((m, h + 5, d), seed)[:, 2:2 + h]
    return lu.randn((h, m, d), seed).transpose(0, 1)  # rows within heads


@pytest.mark.parametrize("d,rotary", [(128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("m,h,kv,layout", [(1, 2, 2, "rows"), (7, 8, 1, "wide"), (33, 6, 3, "heads"), (130, 32, 8, "wide"),
                                           (1000, 4, 4, "rows")])
def test_head_norm_rope(d, rotary, neighbours, m, h, kv, layout):
    q, k = _heads(m, h, d, 1, layout), _heads(m, kv, d, 2, layout)
    table = lu.rope_table(777, rotary)
    pos = torch.randint(777, (m,), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(m))
    desc = dllm.layer_desc(max(64, h * d), h, d, 1e4, 1e-6)
    pairs = dllm.DLLM_ROPE_NEIGHBOURS if neighbours else dllm.DLLM_ROPE_HALVES
    gains = [lu.randn((d,), 3, 0.5), lu.randn((d,), 4, 0.5)]
    for qg, kg in ((gains[0], gains[1]), (None, None), (None, gains[1])):
        error = ints([0])
        qo, ko = torch.zeros_like(q), torch.zeros(m, kv, d, dtype=torch.bfloat16, device="cuda")
        dllm.dllm_head_norm_rope(desc, q, qo, k, ko, pos, table, qg, kg, pairs, error)
        for x, g, out in ((q, qg, qo), (k, kg, ko)):
            want, off = lu.head_norm_rope(x, g, pos, table, rotary, neighbours, 1e-6)
            err = (out.double() - want).abs()
            assert (err <= off).all(), (err / off).max().item()
        q2, k2 = q.clone(memory_format=torch.preserve_format), k.clone()
        dllm.dllm_head_norm_rope(desc, q2, q2, k2, k2, pos, table, qg, kg, pairs, error)  # in place
        assert torch.equal(q2, qo) and torch.equal(k2, ko) and error.item() == 0
        qo2 = torch.zeros_like(q)
        dllm.dllm_head_norm_rope(desc, q, qo2, None, None, pos, table, qg, None, pairs, error)  # queries alone
        assert torch.equal(qo2, qo)


def test_head_norm_rope_leaves_rows_without_a_position():
    m, h, kv, d = 50, 4, 2, 128
    q, k = lu.randn((m, h, d), 1), lu.randn((m, kv, d), 2)
    table = lu.rope_table(64, d)
    pos = [i % 64 if i % 3 else -1 for i in range(m)]
    pos[10], pos[20], pos[40] = 64, -2, 1 << 30
    desc = dllm.layer_desc(h * d, h, d, 1e4)
    for bad in (True, False):
        p = ints(pos if bad else [x if -1 <= x < 64 else -1 for x in pos])
        error, qo, ko = ints([0]), torch.full_like(q, 3.0), torch.full_like(k, 3.0)
        dllm.dllm_head_norm_rope(desc, q, qo, k, ko, p, table, error=error)
        assert error.item() == (dllm.DLLM_DEVERR_BAD_SHAPE if bad else 0)
        for i, x in enumerate(pos):
            there = 0 <= x < 64
            assert there or ((qo[i] == 3.0).all() and (ko[i] == 3.0).all())
            assert not there or not (qo[i] == 3.0).all()


def test_head_norm_rope_rows_of_zeros_large_and_not_finite_values():
    d = 128
    q = lu.randn((6, 2, d), 1)
    q[0] = 0
    q[1] *= 1e4
    q[2] *= 1e-4
    q[3, 0, 5] = math.nan
    q[4, 1, 100] = math.inf
    gain, table, pos = lu.randn((d,), 2), lu.rope_table(10, 64), ints([0, 1, 2, 3, 4, 5])
    out = torch.zeros_like(q)
    desc = dllm.layer_desc(2 * d, 2, d, 1e4, 1e-6)
    dllm.dllm_head_norm_rope(desc, q, out, None, None, pos, table, gain)
    want, off = lu.head_norm_rope(q, gain, pos, table, 64, False, 1e-6)
    fine = [(0, 0), (0, 1), (1, 0), (1, 1), (2, 0), (2, 1), (3, 1), (4, 0), (5, 0), (5, 1)]
    for i, h in fine:
        assert ((out[i, h].double() - want[i, h]).abs() <= off[i, h]).all()
    assert torch.isnan(out[3, 0]).all() and not torch.isfinite(out[4, 1]).all()
    dllm.dllm_head_norm_rope(desc, q, out, None, None, pos, table)  # without a norm: elements behind the rotation as they are
    assert torch.equal(out[4, :, 64:], q[4, :, 64:]) and torch.equal(out[0], q[0])


# ------------------------------------------------------------------ token scores
def _scores(x, tokens, top, scale, some=True):
    m = x.shape[0]
    error = ints([0])
    f = lambda *s: torch.full(s, 9.0, device="cuda")  # noqa: E731
    lse, entropy, logp = f(m), f(m), f(m)
    ids = torch.full((m, top), -9, dtype=torch.int32, device="cuda") if top else None
    best = f(m, top) if top else None
    dllm.dllm_token_scores(x, tokens, logp, lse, entropy, ids, best, scale, error)
    return (lse, entropy, logp, ids, best), error.item()


def _tokens(m, v, seed=0):
    return torch.randint(-1, v, (m,), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(seed))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v,pad", [(1, 1, 0), (3, 2, 1), (5, 7, 0), (4, 64, 3), (17, 1000, 1), (2, 4099, 0), (400, 515, 2),
                                     (1, 126464, 0), (2, 126464, 8), (9, 50001, 7), (40, 126464, 0), (700, 8200, 5)])
def test_token_scores(dtype, m, v, pad):
    x = lu.randn((m, v + pad), m + v, 3.0, dtype)[:, :v]
    for top in (0, 1, 2, 20, 32):
        tokens = _tokens(m, v, top)
        got, bits = _scores(x, tokens, top, 1.0)
        assert bits == 0
        lu.assert_scores(got, x, tokens, top, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-6, 0.01, 0.25, 1.5, 40.0, 50.0, 1e4])
def test_token_scores_at_a_temperature(dtype, scale):
    x = lu.randn((20, 3001), 1, 4.0, dtype)
    tokens = _tokens(20, 3001)
    got, bits = _scores(x, tokens, 5, scale)
    assert bits == 0
    lu.assert_scores(got, x, tokens, 5, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v", [130, 9000, 126464])
def test_token_scores_under_masks(dtype, v):
    """-inf, the type's lowest value, next to nothing left, nothing left, and rows of one value."""
    lowest = torch.finfo(dtype).min
    x = lu.randn((22, v), v, 3.0, dtype)
    u = torch.rand(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[0].masked_fill_(u[0] < 0.9, -math.inf)
    x[1].masked_fill_(u[1] < 0.9, lowest)
    x[2] = -math.inf
    x[3] = lowest
    x[4] = -math.inf
    x[4, v - 1] = 2.0
    x[5] = -math.inf
    x[5, [0, 7, v // 2]] = lowest
    x[6] = lowest
    x[6, v // 3] = -5.0
    x[7] = 0.0
    x[8] = -0.0
    x[8, ::2] = 0.0
    x[9] = -1e30
    x[10] = torch.linspace(-20, 20, v, device="cuda")
    x[11] = torch.linspace(20, -20, v, device="cuda")
    for i, low in enumerate((-1e4, -1e5, -1e9, -1e10, -1e20)):  # finite masks, in front of what is left
        x[13 + i, :v - 20] = low
    x[18], x[19] = x[18] * 1e4, x[19] * 1e20  # large logits
    x[20] = x[20] - 3e4
    x[21, 5] = 2e4
    tokens = _tokens(22, v)
    tokens[6] = v // 3
    for top in (1, 20, 32):
        got, bits = _scores(x, tokens, top, 1.0)
        assert bits == 0
        lu.assert_scores(got, x, tokens, top, 1.0)


@pytest.mark.parametrize("dtype,step", [(torch.bfloat16, 1), (torch.float32, 1), (torch.bfloat16, 8), (torch.float32, 4)])
def test_token_scores_with_the_largest_anywhere(dtype, step):
    """The largest values side by side, in every n-th place for many n (all of them one thread's, for some), and equal."""
    v = 40000
    places = [1, 8, 64, 128, 256, 512, 1024, 2048, 4096, 8192, 16384]
    x = lu.randn((2 * len(places), v), 3, 1.0, dtype)
    for i, n in enumerate(places):
        at = (torch.arange(40000 // max(n, 100), device="cuda") * n + 3 * step) % v
        x[2 * i, at] = 30.0 + (torch.arange(at.numel(), device="cuda") % 50).to(dtype)
        x[2 * i + 1, at] = 30.0
    tokens = _tokens(x.shape[0], v)
    for top in (1, 5, 32):
        got, bits = _scores(x, tokens, top, 1.0)
        assert bits == 0
        lu.assert_scores(got, x, tokens, top, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v", [(6, 1003), (6, 126464), (900, 2000)])
def test_token_scores_of_rows_that_are_not_numbers(dtype, m, v):
    x = lu.randn((m, v), 1, 3.0, dtype)
    x[1, v // 2] = math.nan
    x[2, v - 1] = math.inf
    x[3, 0] = math.nan
    x[3, 1:] = -math.inf
    tokens = _tokens(m, v)
    tokens[1] = -1
    tokens[4] = v
    tokens[5] = v - 1
    (lse, entropy, logp, ids, best), bits = _scores(x, tokens, 4, 1.0)
    assert bits == dllm.DLLM_DEVERR_RANGE | dllm.DLLM_DEVERR_BAD_SHAPE
    for t in (lse, entropy, logp, best):
        assert torch.isnan(t[1:4]).all()
    assert (ids[1:4] == -1).all() and torch.isnan(logp[4]) and torch.isfinite(lse[4])
    keep = [0] + list(range(5, m))
    lu.assert_scores([t[keep] for t in (lse, entropy, logp, ids, best)], x[keep], tokens[keep], 4, 1.0)


def test_token_scores_some_outputs_alone():
    x, tokens = lu.randn((8, 5000), 1, 3.0), _tokens(8, 5000)
    (lse, entropy, logp, ids, best), _ = _scores(x, tokens, 3, 1.0)
    a, b, c, i, t = (torch.zeros_like(y) for y in (lse, entropy, logp, ids, best))
    dllm.dllm_token_scores(x, lse=a)
    dllm.dllm_token_scores(x, entropy=b)
    dllm.dllm_token_scores(x, tokens, c)
    dllm.dllm_token_scores(x, top_ids=i, top_logp=t)
    for got, want in ((a, lse), (b, entropy), (c, logp), (i, ids), (t, best)):
        assert torch.equal(got, want)


def test_token_scores_rows_beyond_32_bits_of_elements():
    v, m = 126464, 17200  # 2.18 G elements
    x = torch.zeros(m, v, dtype=torch.bfloat16, device="cuda")
    x[-3:] = lu.randn((3, v), 1, 3.0)
    tokens = _tokens(m, v)
    got, bits = _scores(x, tokens, 3, 1.0)
    assert bits == 0
    lu.assert_scores([t[-5:] for t in got], x[-5:], tokens[-5:], 3, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v,top", [(3000, 130, 32), (1300, 1001, 20), (700, 4100, 4), (2100, 33, 5), (650, 1000, 20)])
def test_token_scores_of_many_short_rows(dtype, m, v, top):
    x = lu.randn((m, v + 3), m, 3.0, dtype)[:, :v]
    x[5] = -math.inf
    x[6] = torch.finfo(dtype).min
    x[7, 1:] = -math.inf
    x[8] = 1.5
    x[9, ::2] = -1e9
    x[10] = x[10] * 1e5
    tokens = _tokens(m, v)
    got, bits = _scores(x, tokens, top, 1.0)
    assert bits == 0
    lu.assert_scores(got, x, tokens, top, 1.0)


@pytest.mark.parametrize("n,pad", [(500, 0), (501, 0), (502, 2), (503, 1), (504, 0), (257, 6), (193, 0), (130, 1)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_rows_on_any_boundary(n, pad, gated):
    """Rows of y and the residual that begin anywhere, in tiles that end anywhere, into y and in place."""
    c = Linear(1300, 128, n, "silu", gated, bias=True, residual=True, pad=pad, seed=n + pad)
    c.call()
    c.check()
    before = c.residual.clone()
    whole = torch.full((1300, n + pad + 1), 7.0, dtype=torch.bfloat16, device="cuda")
    y = whole[:, 1:n + 1]
    y.copy_(before)
    dllm.dllm_linear(c.desc, c.x, c.w, y, bias=c.bias, residual=y)
    c.check(y, before)
    assert (whole[:, n + 1:] == 7.0).all() and (whole[:, 0] == 7.0).all()


# ------------------------------------------------------------------ together
def test_a_captured_step_of_a_layer_of_grouped_heads():
    """Plan, projection, heads' norm and rotation in place, cache write, attention, output projection, gated feed-forward
    block, head and scores: captured once, replayed while requests grow, end and come.  Each stage against its 64-bit form on
    what the stage before it left."""
    import random

    kv, H, d, D, F, V, batch, width, P = 2, 8, 128, 512, 640, 1003, 5, 12, 30
    r = random.Random(7)
    dev = {k: ints([0] * batch) for k in ("n", "start", "rows", "held", "held_out")}
    dev.update(table=ints([[0] * 8] * batch), cub=ints([0] * (batch + 1)), cus=ints([0] * (batch + 1)), err=ints([0]))
    ring, cap = dllm.PageRing.full(P), batch * width
    pos = ints([-1] * cap)
    view = dllm.BatchView(dev["table"], dev["n"], dev["start"], dev["rows"], dev["cub"], dev["cus"], cap, batch * 512, width, 512,
                          dev["err"])
    kv8 = dllm.Kv8Cache(P, kv, d)
    desc = dllm.layer_desc(D, H, d, 1e4)
    w = {k: lu.randn(s, 20 + i, 1 / math.sqrt(s[1])) for i, (k, s) in enumerate(dict(
        qkv=((H + 2 * kv) * d, D), o=(D, H * d), gu=(2 * F, D), down=(D, F), head=(V, D)).items())}
    bias, gains = lu.randn(((H + 2 * kv) * d,), 30, 0.2), [(1 + lu.randn((D,), 31 + i, 0.2).float()).bfloat16() for i in range(3)]
    q_gain, k_gain = lu.randn((d,), 40), lu.randn((d,), 41)
    table = dllm_table(d, 512)
    lay = dict(qkv=dllm.linear_desc(D, (H + 2 * kv) * d), o=dllm.linear_desc(H * d, D), down=dllm.linear_desc(F, D),
               gu=dllm.linear_desc(D, F, dllm.DLLM_ACT_SILU, True), head=dllm.linear_desc(D, V))
    ws = dllm.workspace(max(dllm.dllm_linear_workspace_size(lay[k], cap, True) for k in ("qkv", "gu", "head")))
    ws_att = dllm.workspace(dllm.dllm_kv8_attention_workspace_size(desc, view.c, kv8.c))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, qkv, raw, o, h1, a, h2, logits = (bf(cap, n) for n in (D, (H + 2 * kv) * d, (H + 2 * kv) * d, H * d, D, F, D, V))
    heads = qkv.view(cap, H + 2 * kv, d)
    q, k, v = heads[:, :H], heads[:, H:H + kv], heads[:, H + kv:]
    lse = torch.zeros(cap, H, device="cuda")
    tokens, ids = ints([0] * cap), torch.zeros(cap, 4, dtype=torch.int32, device="cuda")
    logp, row_lse, entropy, best = (torch.zeros(s, device="cuda") for s in ((cap,), (cap,), (cap,), (cap, 4)))

    def step():
        dllm.dllm_batch_plan(view.c, dev["held"], dev["held_out"], dev["table"], dev["cub"], dev["cus"], ring.c, row_pos=pos)
        dllm.dllm_linear(lay["qkv"], x, w["qkv"], qkv, rms_gain=gains[0], bias=bias, ws=ws, error=dev["err"])
        raw.copy_(qkv)
        dllm.dllm_head_norm_rope(desc, q, q, k, k, pos, table, q_gain, k_gain, error=dev["err"])
        dllm.dllm_kv8_write(desc, view.c, k, v, kv8.c)
        dllm.dllm_kv8_attention(desc, view.c, q, kv8.c, o.view(cap, H, d), lse, ws_att)
        dllm.dllm_linear(lay["o"], o, w["o"], h1, residual=x, error=dev["err"])
        dllm.dllm_linear(lay["gu"], h1, w["gu"], a, rms_gain=gains[1], ws=ws, error=dev["err"])
        dllm.dllm_linear(lay["down"], a, w["down"], h2, residual=h1, error=dev["err"])
        dllm.dllm_linear(lay["head"], h2, w["head"], logits, rms_gain=gains[2], ws=ws, error=dev["err"])
        dllm.dllm_token_scores(logits, tokens, logp, row_lse, entropy, ids, best, error=dev["err"])
        dev["held"].copy_(dev["held_out"])
        ring.state.copy_(ring.state_out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()  # nothing planned yet
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    def near(got, want_off):
        assert ((got.double() - want_off[0]).abs() <= want_off[1]).all()

    n = [0] * batch
    for i in range(6):
        new = [r.choice([1, r.randint(0, width)]) for _ in range(batch)]
        n = [0 if r.random() < 0.1 else y for y in n]
        start, n = n, [y + c for y, c in zip(n, new)]
        for key, val in (("n", n), ("start", start), ("rows", new)):
            dev[key].copy_(ints(val))
        x.copy_(lu.randn((cap, D), 100 + i))
        tokens.copy_(_tokens(cap, V, i))
        graph.replay()
        torch.cuda.synchronize()
        assert dev["err"].item() == 0
        M = sum(new)
        assert pos.tolist() == [s + j for s, c in zip(start, new) for j in range(c)] + [-1] * (cap - M)
        near(raw, lu.linear(x, w["qkv"], gains[0], bias))
        before = raw.view(cap, H + 2 * kv, d)
        near(q[:M], lu.head_norm_rope(before[:M, :H], q_gain, pos[:M], table, d, False, 1e-5))
        near(k[:M], lu.head_norm_rope(before[:M, H:H + kv], k_gain, pos[:M], table, d, False, 1e-5))
        assert torch.equal(heads[M:], before[M:]) and torch.equal(v, before[:, H + kv:])
        b = Batch([1], [0], [1])
        b.n, b.start, b.rows, b.table, b.M = n, start, new, dev["table"].tolist(), cap
        assert_attention(b, q, kv8, o.view(cap, H, d), lse)
        near(h1, lu.linear(o, w["o"], residual=x))
        near(a, lu.linear(h1, w["gu"], gains[1], name="silu", gated=True))
        near(h2, lu.linear(a, w["down"], residual=h1))
        near(logits, lu.linear(h2, w["head"], gains[2]))
        lu.assert_scores((row_lse, entropy, logp, ids, best), logits, tokens, 4, 1.0)


def dllm_table(d, positions):
    """cos and sin as the library makes them."""
    table = torch.zeros(positions, d // 2, 2, device="cuda")
    dllm.dllm_rope_table_build(dllm.layer_desc(128, 128 // d, d, 1e4), positions, table)
    assert (table - lu.rope_table(positions, d)).abs().max() < 1e-6
    return table


def test_scores_of_the_block_heads_logits():
    """Beside dllm_block_lm_head: its log-sum-exp, argmax and confidence are of the logits before their rounding to bf16 (off
    by at most 2^-8 of the largest); the scores' are of the rounded ones."""
    n, D, V = 40, 256, 1000
    lay = dllm.BatchLayout([[0]], [n], [8], [32])
    desc = dllm.layer_desc(D, 2, 128, 1e4)
    h, w, gain = lu.randn((n, D), 1), lu.randn((V, D), 2, 0.2), torch.ones(D, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(32, V, dtype=torch.bfloat16, device="cuda")
    lse, arg, p = torch.zeros(32, device="cuda"), ints([0] * 32), torch.zeros(32, device="cuda")
    ws = dllm.workspace(dllm.dllm_lm_head_workspace_size(desc, lay.c, V))
    dllm.dllm_block_lm_head(desc, lay.c, V, h, gain, w, logits, lse, arg, p, ws)
    (lse2, _, logp, ids, best), bits = _scores(logits, arg, 2, 1.0)
    assert bits == 0
    lu.assert_scores((lse2, None, logp, ids, best), logits, arg, 2, 1.0)
    off = lu.HALF_BF16 * logits.float().abs().amax(1) + 1e-4
    assert ((lse - lse2).abs() <= off).all() and ((p.log() - logp).abs() <= 2 * off).all()


def test_heads_of_many_rows_in_place():
    m, h, kv, d = 6001, 8, 2, 128
    buf = lu.randn((m, h + 2 * kv, d), 1)
    q, k, before = buf[:, :h], buf[:, h:h + kv], buf.clone()
    table, gains, error = lu.rope_table(500, d), [lu.randn((d,), 3, 0.5), lu.randn((d,), 4, 0.5)], ints([0])
    pos = torch.arange(m, device="cuda", dtype=torch.int32) % 500
    pos[5::97] = -1
    dllm.dllm_head_norm_rope(dllm.layer_desc(h * d, h, d, 1e4, 1e-6), q, q, k, k, pos, table, *gains, error=error)
    there = pos >= 0
    for got, x, g in ((q, before[:, :h], gains[0]), (k, before[:, h:h + kv], gains[1])):
        want, off = lu.head_norm_rope(x[there], g, pos[there], table, d, False, 1e-6)
        assert ((got[there].double() - want).abs() <= off).all()
    assert torch.equal(buf[~there], before[~there]) and torch.equal(buf[:, h + kv:], before[:, h + kv:])
    assert error.item() == 0


class Chain:
    """A few rows' product, the heads and the scores of one request, each with buffers of its own."""

    def __init__(self, m, seed):
        self.lin = Linear(m, 1024, 10 * 128, norm=True, bias=True, seed=seed)
        self.heads = self.lin.y.view(m, 10, 128)
        self.out = torch.zeros_like(self.heads)
        self.pos = torch.arange(m, device="cuda", dtype=torch.int32) + seed
        self.table, self.gain = lu.rope_table(64, 128), lu.randn((128,), seed + 7, 0.5)
        self.desc = dllm.layer_desc(8 * 128, 8, 128, 1e4, 1e-6)
        self.logits, self.tokens = self.out.view(m, 1280), _tokens(m, 1280, seed)
        self.f = [torch.zeros(m, device="cuda") for _ in range(3)]
        self.ids, self.best = torch.zeros(m, 4, device="cuda", dtype=torch.int32), torch.zeros(m, 4, device="cuda")

    def call(self):
        self.lin.call()
        dllm.dllm_head_norm_rope(self.desc, self.heads[:, :8], self.out[:, :8], self.heads[:, 8:], self.out[:, 8:], self.pos,
                                 self.table, self.gain, self.gain, error=self.lin.error)
        dllm.dllm_token_scores(self.logits, self.tokens, *self.f, self.ids, self.best, 1.0, self.lin.error)

    def results(self):
        assert self.lin.error.item() == 0
        return [t.clone() for t in (self.lin.y, self.out, *self.f, self.ids, self.best)]


@pytest.mark.parametrize("m", [1, 2, 5])
def test_calls_on_two_streams_at_once_and_captured(m):
    cs = [Chain(m, s) for s in (1, 2)]
    xs = [c.lin.x.clone() for c in cs]
    want = {}
    for i, c in enumerate(cs):  # each of the rows through each of the chains, one call behind the other
        for j, x in enumerate(xs):
            c.lin.x.copy_(x)
            c.call()
            torch.cuda.synchronize()
            want[i, j] = c.results()
            c.lin.check()
    streams = [torch.cuda.Stream() for _ in cs]
    for turn in range(6):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                c.lin.x.copy_(xs[(i + turn) % 2])
                c.call()
        torch.cuda.synchronize()
        for i, c in enumerate(cs):
            assert all(torch.equal(a, b) for a, b in zip(c.results(), want[i, (i + turn) % 2]))
    graphs = [torch.cuda.CUDAGraph() for _ in cs]
    for c, g in zip(cs, graphs):
        with torch.cuda.graph(g):
            c.call()
    for turn in range(4):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                c.lin.x.copy_(xs[(i + turn) % 2])
                graphs[i].replay()
        torch.cuda.synchronize()
        for i, c in enumerate(cs):
            assert all(torch.equal(a, b) for a, b in zip(c.results(), want[i, (i + turn) % 2]))
