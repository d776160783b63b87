"""Where a layer's calls can go wrong unseen by one thread's products with random weights."""
import ctypes
import math
import threading

import pytest
import torch

import layer_util as lu
from block_wise_kv_gb300 import dllm
from kv8_util import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_wise_kv_gb300 import build

    build.build()
    dllm.load()
    torch.cuda.init()


# ------------------------------------------------------------------ two host threads
def _raw(desc, x, w, y, error, stream):
    """The C call and its arguments, so that little but the call itself holds two threads apart."""
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    args = (ctypes.byref(desc), x.shape[0], p(x), x.shape[1], None, p(w), None, None, y.shape[1], p(y), y.shape[1], p(error),
            None, 0, ctypes.c_void_p(stream.cuda_stream))
    return lambda: dllm.load().dllm_linear(*args)


def _together(*works):
    """Each on a thread of its own; what they raise is raised here."""
    wrong, gate = [], threading.Barrier(len(works))

    def run(work):
        gate.wait()
        try:
            work()
        except BaseException as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if wrong:
        raise wrong[0]


def test_a_host_threads_first_call_is_a_product():
    """Nothing before it has made the device's context the thread's own."""
    m, k, n = 48, 256, 384
    x, w, y, error = lu.randn((m, k), 1), lu.randn((n, k), 2, 1 / math.sqrt(k)), lu.randn((m, n), 3), ints([0])
    stream, status = torch.cuda.Stream(), []
    call = _raw(dllm.linear_desc(k, n), x, w, y, error, stream)
    torch.cuda.synchronize()
    _together(lambda: status.append(call()))
    torch.cuda.synchronize()
    want, off = lu.linear(x, w)
    assert status == [dllm.DLLM_OK] and ((y.double() - want).abs() <= off).all() and error.item() == 0


@pytest.mark.parametrize("sizes", [((64, 4096, 4096), (16, 256, 768)), ((64, 1024, 256), (3, 64, 128))])
def test_two_host_threads_call_products_of_one_activation(sizes):
    """Their kernels take different amounts of shared memory, on two streams."""
    works = []
    for i, (m, k, n) in enumerate(sizes):
        x, w, y, error = lu.randn((m, k), i), lu.randn((n, k), 10 + i, 1 / math.sqrt(k)), lu.randn((m, n), 20), ints([0])
        stream, want = torch.cuda.Stream(), lu.linear(x, w)
        call = _raw(dllm.linear_desc(k, n), x, w, y, error, stream)

        def work(call=call, y=y, error=error, stream=stream, want=want):
            with torch.cuda.stream(stream):
                for turn in range(4000):
                    assert call() == dllm.DLLM_OK, turn
                    if turn % 500 == 499:
                        assert ((y.double() - want[0]).abs() <= want[1]).all() and error.item() == 0
                        y.fill_(7.0)

        works.append(work)
    torch.cuda.synchronize()
    _together(*works)


# ------------------------------------------------------------------ long waits
def test_rows_so_long_that_a_product_takes_most_of_a_second():
    """2^30 columns, all but some of them zero: the sums are exact, and whoever makes y waits for all of it."""
    k, m = 1 << 30, 3
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, k, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 63, 64, 12345, k // 8 - 1, k // 8, k // 2 + 7, k - 65, k - 64, k - 1], device="cuda")
    x[:, at] = torch.arange(1, 1 + m * at.numel(), device="cuda").view(m, -1).bfloat16()
    w[0, at] = torch.arange(at.numel(), device="cuda").bfloat16() - 4
    y, error = torch.zeros(m, 1, dtype=torch.bfloat16, device="cuda"), ints([0])
    dllm.dllm_linear(dllm.linear_desc(k, 1), x, w, y, error=error)
    want = (x[:, at].double() * w[0, at].double()).sum(1, keepdim=True)
    assert error.item() == 0 and torch.equal(y, want.bfloat16()), (error.item(), y, want)


# ------------------------------------------------------------------ the normed rows themselves
@pytest.mark.parametrize("m,k,at_a_time", [
    (512, 4096, 1), (512, 4096, 2), (256, 8200, 1),                       # one or two rows
    (4000, 256, 8), (1500, 1000, 5),                                      # normed inside the product
    (1500, 1024, 1500), (1200, 1032, 1200), (600, 4096, 600), (300, 4104, 300), (100, 8448, 100)])  # by the norm's kernel
@pytest.mark.parametrize("size", [1.0, 1e-4, 3e4])
def test_normed_rows_are_the_nearest_bf16(m, k, at_a_time, size):
    """With the identity for a weight y is x^ itself.  One value in some 40000 lies within a 32-bit step of the middle of two
    bf16 values, where a product in 32 bits alone rounds the wrong way."""
    eps = 2.0 ** -17  # the same in 32 and 64 bits
    x, gain = lu.randn((m, k), k, size), (1 + lu.randn((k,), 2, 0.3).float()).bfloat16()
    eye = torch.eye(k, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    desc = dllm.linear_desc(k, k, rms_eps=eps)
    ws = dllm.workspace(dllm.dllm_linear_workspace_size(desc, at_a_time, True))
    for i in range(0, m, at_a_time):
        dllm.dllm_linear(desc, x[i:i + at_a_time], eye, y[i:i + at_a_time], rms_gain=gain, ws=ws)
    want = lu.nearest_bf16(lu.rms_norm(x, gain, eps))
    assert torch.equal(y.double(), want), ((y.double() != want).sum().item(), y.numel())


# ------------------------------------------------------------------ the activations' tails
ACTS = [("silu", dllm.DLLM_ACT_SILU), ("gelu", dllm.DLLM_ACT_GELU), ("gelu_tanh", dllm.DLLM_ACT_GELU_TANH)]


def _act(t, name):
    """(value, how far it lies down the tail: z of its e^-z) in 64 bits, without a difference of near numbers."""
    if name == "gelu":
        return 0.5 * t * torch.erfc(-t * math.sqrt(0.5)), t.clamp(max=0) ** 2 / 2
    u = t if name == "silu" else 2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)
    return t * torch.sigmoid(u), (-u).clamp(min=0)


def _assert_act(y, t, name):
    """Relative to the value: bf16's rounding; the exponent z of e^-z comes of a handful of roundings of 2^-24 of it, which are
    that much of the value; the functions' own error and the last products are counted as 2^-19.  Below bf16's normal range:
    one of its steps there, 2^-133."""
    want, z = _act(t, name)
    off = (lu.HALF_BF16 + 2.0 ** -21 * (4 + z)) * want.abs() + 2.0 ** -133
    bad = ((y.double() - want).abs() <= off).logical_not().nonzero()[:4].tolist()
    assert not bad, [(t.expand_as(y)[i, j].item(), y[i, j].item(), want.expand_as(y)[i, j].item()) for i, j in bad]


@pytest.mark.parametrize("name,act", ACTS)
@pytest.mark.parametrize("m", [1, 2, 40, 6000])
def test_activations_keep_their_tails(name, act, m):
    """One 1 in each row of W: t is the chosen value without any rounding.  Every bf16 value from -104 to 104, some beyond."""
    u = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    t = torch.cat([u[(u.abs() <= 104)], torch.tensor([-3e38, -1e20, -1e5, 1e5, 1e20, 3e38], device="cuda").bfloat16()])
    assert t.numel() > 33000
    if m <= 2:  # the values are W's
        x = torch.zeros(m, 8, dtype=torch.bfloat16, device="cuda")
        x[:, 0] = 1
        w = torch.zeros(t.numel(), 8, dtype=torch.bfloat16, device="cuda")
        w[:, 0] = t
        y = torch.zeros(m, t.numel(), dtype=torch.bfloat16, device="cuda")
        dllm.dllm_linear(dllm.linear_desc(8, t.numel(), act), x, w, y)
        _assert_act(y, t.double()[None], name)
        return
    n = 96 if m == 40 else 520
    w = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1
    for part in t.split(m):
        x = torch.zeros(part.numel(), 8, dtype=torch.bfloat16, device="cuda")
        x[:, 0] = part
        y = torch.zeros(part.numel(), n, dtype=torch.bfloat16, device="cuda")
        dllm.dllm_linear(dllm.linear_desc(8, n, act), x, w, y)
        _assert_act(y, part.double()[:, None], name)


# ------------------------------------------------------------------ the kernel in front
@pytest.mark.parametrize("m", [1, 2, 64, 1500])
def test_products_of_what_the_librarys_kernel_in_front_wrote(m):
    """Rows, weight, bias and residual each by a call of this library directly in front (which lets its successor start
    early), calls one behind the other without a wait; other values every turn."""
    k, n, turns = 1024, 640, 24
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    table, pos = lu.rope_table(64, 128), torch.arange(m, device="cuda", dtype=torch.int32) % 64
    srcs = [dict(x=lu.randn((m, k), s), w=lu.randn((n, k), s + 1), z=lu.randn((1, k), s + 2)) for s in (1, 11)]
    wk, wn, wnn = lu.randn((k, k), 5, 1 / 32), lu.randn((n, k), 6, 1 / 32), lu.randn((n, n), 9, 1 / 25)
    gain = (1 + lu.randn((k,), 7, 0.2).float()).bfloat16()
    h, w, bias, r, turned = bf(m, k), bf(n, k), bf(1, n), bf(m, n), bf(m, n)
    tokens, error = _tokens(m, n), ints([0])
    square, out = dllm.linear_desc(k, k), dllm.linear_desc(k, n)
    heads = dllm.layer_desc(n, n // 128, 128, 1e4)
    ws = dllm.workspace(dllm.dllm_linear_workspace_size(out, m, True))

    def turn(s, ys, logp):
        dllm.dllm_linear(square, s["w"], wk, w, error=error)
        dllm.dllm_linear(square, s["x"], wk, h, error=error)
        dllm.dllm_linear(out, h, w, ys[0], error=error)                                  # rows in front, the weight before
        dllm.dllm_linear(out, s["z"], wn, bias, error=error)
        dllm.dllm_linear(out, h, wn, ys[1], bias=bias[0], error=error)                   # bias in front
        dllm.dllm_linear(out, h, wn, r, rms_gain=gain, ws=ws, error=error)               # (the norm's kernel in front)
        dllm.dllm_linear(out, s["x"], w, ys[2], residual=r, error=error)                 # residual in front
        dllm.dllm_linear(out, s["x"], wn, ys[3], rms_gain=gain, ws=ws, error=error)      # the workspace once more
        dllm.dllm_head_norm_rope(heads, ys[3].view(m, n // 128, 128), turned.view(m, n // 128, 128), None, None, pos, table,
                                 error=error)
        dllm.dllm_linear(dllm.linear_desc(n, n), turned, wnn, ys[4], residual=turned, error=error)
        dllm.dllm_linear(square, s["w"], wk, w, error=error)
        dllm.dllm_linear(out, s["x"], w, ys[5], error=error)                             # the weight in front
        dllm.dllm_token_scores(ys[5], tokens, logp, error=error)

    want = []
    for s in srcs:
        ys, logp = [bf(m, n) for _ in range(6)], torch.zeros(m, device="cuda")
        for _ in range(2):
            turn(s, ys, logp)
            torch.cuda.synchronize()
        want.append(ys + [logp])
    got = [([bf(m, n) for _ in range(6)], torch.zeros(m, device="cuda")) for _ in range(turns)]
    torch.cuda.synchronize()
    for i, (ys, logp) in enumerate(got):
        turn(srcs[i % 2], ys, logp)
    torch.cuda.synchronize()
    assert error.item() == 0
    for i, (ys, logp) in enumerate(got):
        for j, (a, b) in enumerate(zip(ys + [logp], want[i % 2])):
            assert torch.equal(a, b), (i, j)
    ok, off = lu.linear(srcs[(turns - 1) % 2]["x"], w)
    assert ((got[-1][0][5].double() - ok).abs() <= off).all()


def _tokens(m, v):
    return torch.arange(m, device="cuda", dtype=torch.int32) % v


# ------------------------------------------------------------------ logits as far apart as their type holds
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,v", [(3, 37), (3, 5003), (2, 126464), (700, 300)])
@pytest.mark.parametrize("scale", [2e-38, 1e-37, 1e-3, 0.25, 1.0])
def test_token_scores_of_logits_whose_difference_is_no_number_of_32_bits(dtype, m, v, scale):
    lowest = torch.finfo(dtype).min
    x = lu.randn((m, v), v, 1e38, dtype).clamp(lowest, -lowest)
    x[0, v // 2], x[0, 1] = -lowest, lowest
    x[1, 2::3] = lowest
    x[1, 0] = 2e38
    tokens = torch.ones(m, dtype=torch.int32, device="cuda")
    tokens[1] = 2
    f = lambda *s: torch.full(s, 9.0, device="cuda")  # noqa: E731
    lse, entropy, logp, ids, best, error = f(m), f(m), f(m), ints([[0] * 32] * m), f(m, 32), ints([0])
    dllm.dllm_token_scores(x, tokens, logp, lse, entropy, ids, best, scale, error)
    assert error.item() == 0
    lu.assert_scores((lse, entropy, logp, ids, best), x, tokens, 32, scale)


def test_token_scores_written_between_the_rows_of_the_logits():
    buf = lu.randn((6, 1100), 1, 3.0)
    x, lse = buf[:, :1000], buf.view(torch.float32)[2, 502:508]
    entropy, ids, best = torch.zeros(6, device="cuda"), ints([[0] * 4] * 6), torch.zeros(6, 4, device="cuda")
    rest = buf.clone()
    dllm.dllm_token_scores(x, lse=lse, entropy=entropy, top_ids=ids, top_logp=best)
    lu.assert_scores((lse, entropy, None, ids, best), x, ints([0] * 6), 4, 1.0)
    rest.view(torch.float32)[2, 502:508] = lse
    assert torch.equal(buf, rest)
