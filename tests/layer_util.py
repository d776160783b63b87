"""Plain 64-bit forms of a layer's products, head norms with rotation and token scores, and the tolerances that go with
them: bf16 rounds by at most 2^-8 of a value, fp32 by 2^-24."""
import math

import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_FP32 = torch.finfo(torch.float32).eps / 2
ACTS = ("none", "silu", "gelu", "gelu_tanh")


def randn(shape, seed, size=1.0, dtype=torch.bfloat16):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=gen) * size).to(dtype)


def nearest_bf16(x):
    """float64 -> the nearest bf16 value (ties to even; normal range), in float64."""
    f, e = torch.frexp(x)
    return torch.ldexp(torch.round(f * 256), e - 8).float().bfloat16().double()  # (ldexp itself is off by a 64-bit step)


def rms_norm(x, gain, eps):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()


def act(t, name):
    if name == "silu":
        return t * torch.sigmoid(t)
    if name == "gelu":
        return 0.5 * t * torch.erfc(-t * math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
    return t


def linear(x, w, gain=None, bias=None, residual=None, name="none", gated=False, eps=1e-5):
    """(y, how far a right kernel's may be off).  The tensor core adds 16 products at a time to an fp32 sum: each addition,
    and each alignment of its products, loses at most 2^-23 (truncation) of the sum of magnitudes S, 2 K / 16 in all.
    silu and both gelus are steeper than 1.13 nowhere; their own evaluation is off by a few fp32 steps, counted as 2^-20 of
    their argument."""
    x = x.double() if gain is None else nearest_bf16(rms_norm(x, gain, eps))
    w = w.double()
    t, s = x @ w.t(), x.abs() @ w.abs().t()
    off = (2 * math.ceil(x.shape[1] / 16) + 2) * 2 * HALF_FP32 * s
    if bias is not None:
        t = t + bias.double()
        off = off + HALF_FP32 * t.abs()
    if gated:
        g, u, og, ou = t[:, 0::2], t[:, 1::2], off[:, 0::2], off[:, 1::2]
        a = act(g, name)
        oa = 1.13 * og + 2.0 ** -20 * g.abs()
        y, off = a * u, oa * u.abs() + a.abs() * ou + oa * ou
    else:
        y, off = act(t, name), 1.13 * off + 2.0 ** -20 * t.abs()
    if residual is not None:
        y = y + residual.double()
    return y, off + (HALF_BF16 + 2 * HALF_FP32) * y.abs() + 1e-30


def head_norm_rope(x, gain, pos, table, rotary, neighbours, eps):
    """(out, how far): rows with a position; fp32 holds every step (about ten roundings of the two elements of a pair, 2^-20
    of them at most), bf16 rounds once."""
    u = x.double() if gain is None else rms_norm(x, gain, eps)
    i = torch.arange(rotary // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if neighbours else (i, i + rotary // 2)
    cs = table.double()[pos.long()][:, None]
    c, s = cs[..., 0], cs[..., 1]
    y, size = u.clone(), u.abs()
    y[..., a], y[..., b] = u[..., a] * c - u[..., b] * s, u[..., a] * s + u[..., b] * c
    size[..., a] = size[..., b] = u[..., a].abs() + u[..., b].abs()
    return y, HALF_BF16 * y.abs() + 2.0 ** -20 * size + 1e-30


def rope_table(positions, rotary, theta=1e4):
    i = torch.arange(rotary // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * theta ** (-2.0 * i / rotary)
    return torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()


def token_scores(logits, tokens, top, scale):
    """lse, entropy, logp, ids, log p of the ids, from the definition, row by row; rows without a token left included."""
    x = logits.double()
    m = x.amax(-1, keepdim=True)
    u = torch.where(x > -math.inf, (x - m) * scale, -math.inf)
    log_s = torch.logsumexp(u, -1, keepdim=True)
    empty = m[:, 0] == -math.inf
    lp = torch.where(empty[:, None], -math.inf, u - log_s)
    p = lp.exp()
    entropy = torch.where(empty, 0.0, -torch.where(p > 0, p * lp, 0.0).sum(-1))
    lse = torch.where(empty, -math.inf, m[:, 0] * scale + log_s[:, 0])
    logp = lp.gather(1, tokens.long().clamp(min=0)[:, None])[:, 0]
    logp = torch.where(tokens < 0, 0.0, logp)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    best = lp.gather(1, order)
    there = x.gather(1, order) > -math.inf
    ids, best = torch.where(there, order, -1), torch.where(there, best, -math.inf)
    if top > ids.shape[1]:
        more = (ids.shape[0], top - ids.shape[1])
        ids = torch.cat([ids, torch.full(more, -1, device=ids.device)], 1)
        best = torch.cat([best, torch.full(more, -math.inf, device=ids.device, dtype=best.dtype)], 1)
    return lse, entropy, logp, ids.int(), best


def assert_scores(got, logits, tokens, top, scale):
    """A weight's exponent is off by 2^-23 of itself (two roundings), ex2 by 2^-22: what the sum has of it is 2^-22 (1 + mean
    exponent), a mean exponent being at most log2 of the vocabulary.  A thread adds up to V / 256 weights one after the other
    and a handful of joins: 2^-24 each.  The same holds for the entropy's second sum, whose terms are up to that mean
    exponent.  Results round by 2^-23 of their size."""
    lse, entropy, logp, ids, best = (None if t is None else t.cpu() for t in got)
    want = [t.cpu() for t in token_scores(logits, tokens, top, scale)]
    v = logits.shape[1]
    bits = math.log2(v) + 1
    off = 2.0 ** -22 * (1 + bits) + (v / 256 + 64) * HALF_FP32
    for name, a, b, extra in (("lse", lse, want[0], 1), ("entropy", entropy, want[1], bits), ("logp", logp, want[2], 1),
                              ("top", best, want[4], 1)):
        if a is None:
            continue
        b32 = b.float()  # beyond fp32's range: infinite
        assert torch.equal(torch.isfinite(a), torch.isfinite(b32)) and torch.equal(a[~torch.isfinite(a)], b32[~torch.isfinite(b32)]), name
        fine = torch.isfinite(b32)
        err = (a.double() - b).abs()[fine]
        most = (off * extra + 4 * HALF_FP32 * b.abs())[fine]
        assert (err <= most).all(), (name, err.max(), (err / most).max())
    if ids is not None:
        assert torch.equal(ids, want[3]), (ids != want[3]).nonzero()[:5]
