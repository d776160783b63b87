"""Cases, inputs, plain forms and 64-bit forms of the operators of a layer of grouped heads, and of its answers.

Three operators that a program with its own projection runs around the 8-bit paged cache:

* ``linear``: a product with a weight, RMSNorm of its rows before it, bias, activation (also of gate and up units side by
  side) and residual after it (``dllm_linear``);
* ``rope``: the norm of each head of the queries and keys and the rotation by position, packed rows, grouped heads
  (``dllm_head_norm_rope``);
* ``scores``: log probabilities of given tokens, log-sum-exp, entropy and the most likely tokens of each row of logits
  (``dllm_token_scores``).

Where ``own`` is false, ``run`` computes them with elementary torch operations in 32 bits; where it is true it makes the
library's calls.
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The smallest call: the query, key and value projection of the repository's tiny workload (d_model 256, a block
        # of 32), where latency counts.
        dict(name="linear_tiny", op="linear", rows=32, k=256, n=768, act="none", gated=False, norm=True, bias=False,
             residual=False, pad=0),
        # One new token: the projection to 32 query, 8 key and 8 value heads, normed, with a bias.  All weights, one row.
        dict(name="linear_token", op="linear", rows=1, k=4096, n=6144, act="none", gated=False, norm=True, bias=True,
             residual=False, pad=0),
        # 64 sequences of single tokens: the attention's output projection, added to the residual stream.
        dict(name="linear_tokens", op="linear", rows=64, k=4096, n=4096, act="none", gated=False, norm=False, bias=False,
             residual=True, pad=0),
        # The blocks of the headline batch (16 x 32 rows): the gated first half of the feed-forward block.
        dict(name="linear_block_gated", op="linear", rows=512, k=4096, n=12288, act="silu", gated=True, norm=True,
             bias=False, residual=False, pad=0),
        # Sizes that fill no tile, rows out of wider ones, everything the epilogue has.
        dict(name="linear_odd", op="linear", rows=777, k=1000, n=1003, act="gelu", gated=False, norm=False, bias=True,
             residual=True, pad=24),
        # Whole prompts (4 x 5120 rows): the second half of the feed-forward block, the longest sums.
        dict(name="linear_prompt", op="linear", rows=20480, k=12288, n=4096, act="none", gated=False, norm=False,
             bias=False, residual=True, pad=0),
        # A batch of single tokens, four query heads to a key head, both normed.
        dict(name="rope_tokens", op="rope", rows=64, none=0, heads=32, kv_heads=8, d=128, rotary=128, pairs="halves",
             norm=True, max_pos=16384),
        # The blocks of the headline batch with half of each head rotated, neighbours paired; some rows without a request.
        dict(name="rope_block", op="rope", rows=512, none=37, heads=32, kv_heads=32, d=128, rotary=64,
             pairs="neighbours", norm=True, max_pos=1536),
        # Whole prompts, queries and keys as they lie in the projection's output.
        dict(name="rope_prompt", op="rope", rows=20480, none=0, heads=32, kv_heads=8, d=128, rotary=128, pairs="halves",
             norm=True, max_pos=5120),
        # One row of logits with 20 alternatives: what an answer's next token costs.
        dict(name="scores_token", op="scores", rows=1, vocab=126464, dtype="bf16", top=20, scale=1.0, masked=0.0, pad=0),
        # The blocks of the headline batch: confidence and margin of every masked position.
        dict(name="scores_block", op="scores", rows=512, vocab=126464, dtype="bf16", top=2, scale=1.0, masked=0.0, pad=0),
        # 32-bit logits of an odd vocabulary under a grammar's mask, a temperature, rows that start anywhere, one with
        # nothing left.
        dict(name="scores_masked", op="scores", rows=333, vocab=32003, dtype="fp32", top=8, scale=0.8, masked=0.7,
             pad=5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rope", "scores"])
    if op == "linear":
        gated = rng.random() < 0.3
        k = 8 * _log_int(rng, 8, 1536)
        n = _log_int(rng, 64, 12288)
        most = 20480 * 12288 * 4096 // (k * n * (2 if gated else 1))
        return dict(op=op, rows=_log_int(rng, 1, max(1, min(20480, most))), k=k, n=n,
                    act=rng.choice(["none", "silu", "gelu", "gelu_tanh"]), gated=gated, norm=rng.random() < 0.4,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 24]))
    if op == "rope":
        d = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8, 32]) * (128 // d)
        heads = kv * rng.choice([1, 2, 4, 8])
        rows = _log_int(rng, 1, min(20480, 20480 * 40 * 128 // ((heads + kv) * d)))
        return dict(op=op, rows=rows, none=rng.randint(0, rows // 4), heads=heads, kv_heads=kv, d=d,
                    rotary=rng.choice([64, d]), pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.7,
                    max_pos=_log_int(rng, 64, 16384))
    dtype = rng.choice(["bf16", "fp32"])
    vocab = _log_int(rng, 1000, 126464)
    rows = _log_int(rng, 1, min(4096, 512 * 126464 // (vocab * (2 if dtype == "fp32" else 1))))
    return dict(op=op, rows=rows, vocab=vocab, dtype=dtype, top=rng.choice([0, 1, 2, 5, 20, 32]),
                scale=rng.choice([1.0, 0.8, 0.5]), masked=rng.choice([0.0, 0.0, 0.7]), pad=rng.choice([0, 0, 1, 5]))


def work(case):
    m = case["rows"]
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        wide = 2 * n if case["gated"] else n
        values = m * k + wide * k + m * n * (2 if case["residual"] else 1)
        return {"bytes": 2 * (values + (wide if case["bias"] else 0) + (k if case["norm"] else 0)), "flops": 2 * m * k * wide}
    if case["op"] == "rope":
        there = m - case["none"]
        rows = there * (case["heads"] + case["kv_heads"]) * case["d"] * 2 * 2
        return {"bytes": rows + min(there, case["max_pos"]) * case["rotary"] * 4 + 4 * m, "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": m * (case["vocab"] * size + 16 + 8 * case["top"]), "flops": 0}


# ------------------------------------------------------------------ inputs
def _rows(m, width, pad, gen, size=1.0):
    """bf16 [m][width], each row out of one that is `pad` longer."""
    x = torch.randn(m, width + pad, device="cuda", generator=gen) * size
    return x.to(torch.bfloat16)[:, :width]


def _table(max_pos, rotary):
    """(cos, sin) of p theta^(-2i / rotary), theta 5e5, formed in 64 bits."""
    i = torch.arange(rotary // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * torch.pow(5e5, -2.0 * i / rotary)
    return torch.stack([torch.cos(angle), torch.sin(angle)], -1).float()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    m = case["rows"]
    s = dict(case=case)
    if case["op"] == "linear":
        k, n, pad = case["k"], case["n"], case["pad"]
        wide = 2 * n if case["gated"] else n
        s["x"] = _rows(m, k, pad, gen)
        s["w"] = _rows(wide, k, 0, gen, 0.02)
        s["gain"] = (1 + 0.1 * torch.randn(k, device="cuda", generator=gen)).to(torch.bfloat16) if case["norm"] else None
        s["bias"] = _rows(1, wide, 0, gen, 0.1)[0] if case["bias"] else None
        s["residual"] = _rows(m, n, pad, gen) if case["residual"] else None
        s["y"] = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "rope":
        h, kv, d = case["heads"], case["kv_heads"], case["d"]
        qkv = _rows(m, (h + 2 * kv) * d, 0, gen).view(m, h + 2 * kv, d)
        s["q"], s["k"] = qkv[:, :h], qkv[:, h:h + kv]
        for name in ("q_gain", "k_gain"):
            s[name] = (1 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(torch.bfloat16) if case["norm"] else None
        # sequences one behind the other, of up to max_pos rows; at the end the rows without a request
        pos = torch.arange(m, device="cuda") + torch.randint(case["max_pos"], (1,), device="cuda", generator=gen)
        s["pos"] = torch.where(torch.arange(m, device="cuda") < m - case["none"], pos % case["max_pos"], -1).to(torch.int32)
        s["table"] = _table(case["max_pos"], case["rotary"])
        s["q_out"] = torch.zeros(m, h, d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(m, kv, d, dtype=torch.bfloat16, device="cuda")
        return s
    v = case["vocab"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x = 2.5 * torch.randn(m, v + case["pad"], device="cuda", generator=gen)
    if case["masked"]:
        u = torch.rand(m, v + case["pad"], device="cuda", generator=gen)
        x.masked_fill_(u < case["masked"], -math.inf)  # what the grammar forbids
        x.masked_fill_(u > 0.97, torch.finfo(dtype).min)  # what another filter has put at the type's lowest value
        x[m // 2] = -math.inf  # a row with nothing left
    s["logits"] = x.to(dtype)[:, :v]
    del x
    # given tokens: any that no mask forbids
    lot = torch.rand(m, v, device="cuda", generator=gen).masked_fill_(s["logits"] < -1e30, -1.0)
    s["tokens"] = lot.argmax(-1).to(torch.int32)
    if m > 8:
        s["tokens"][m - 1] = -1  # a row without a given token
    for name in ("logp", "lse", "entropy"):
        s[name] = torch.zeros(m, device="cuda")
    s["top_ids"] = torch.zeros(m, case["top"], dtype=torch.int32, device="cuda") if case["top"] else None
    s["top_logp"] = torch.zeros(m, case["top"], device="cuda") if case["top"] else None
    return s


# ------------------------------------------------------------------ the plain forms
def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _linear_plain(s):
    case = s["case"]
    x = s["x"].float()
    if case["norm"]:  # the normed rows are bf16 by definition: what a matrix instruction takes
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["gain"].float()
        x = x.to(torch.bfloat16).float()
    t = x @ s["w"].float().t()
    if case["bias"]:
        t = t + s["bias"].float()
    t = _act(t[:, 0::2], case["act"]) * t[:, 1::2] if case["gated"] else _act(t, case["act"])
    if case["residual"]:
        t = t + s["residual"].float()
    s["y"].copy_(t)
    return s["y"]


def _turn(x, cos, sin, pairs):
    """The rotation of the first columns of each head, as many as the table has."""
    r = 2 * cos.shape[-1]
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if pairs == "halves" else (x[..., 0:r:2], x[..., 1:r:2])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([u, v], -1) if pairs == "halves" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _rope_plain(s):
    case = s["case"]
    pos = s["pos"].long()
    there = pos >= 0
    cs = s["table"][pos.clamp(min=0)][:, None]
    for name in ("q", "k"):
        x = s[name].float()
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s[name + "_gain"].float()
        x = _turn(x, cs[..., 0], cs[..., 1], case["pairs"])
        out = s[name + "_out"]
        out.copy_(torch.where(there[:, None, None], x.to(torch.bfloat16), out))
    return {"q": s["q_out"], "k": s["k_out"]}


def _scores_plain(s):
    case = s["case"]
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    u = torch.where(x > -math.inf, (x - top) * case["scale"], -math.inf)  # log of each token's weight
    e = torch.exp(u)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    s["lse"].copy_((top * case["scale"] + log_total)[:, 0])
    empty = total[:, 0] == 0
    mean = torch.where(e > 0, e * u, 0.0).sum(-1) / total[:, 0]
    s["entropy"].copy_(torch.where(empty, 0.0, log_total[:, 0] - mean))
    own_u = u.gather(1, s["tokens"].long().clamp(min=0)[:, None])
    logp = torch.where(empty, -math.inf, (own_u - log_total)[:, 0])
    s["logp"].copy_(torch.where(s["tokens"] >= 0, logp, 0.0))
    if case["top"]:
        best, ids = torch.sort(x, dim=-1, descending=True, stable=True)
        best, ids = best[:, :case["top"]], ids[:, :case["top"]]
        s["top_ids"].copy_(torch.where(best > -math.inf, ids, -1))
        s["top_logp"].copy_(torch.where(best > -math.inf, (best - top) * case["scale"] - log_total, -math.inf))
    return _scores_outputs(s)


def _scores_outputs(s):
    return {k: s[k] for k in ("logp", "lse", "entropy", "top_ids", "top_logp") if s[k] is not None}


# ------------------------------------------------------------------ the library's calls
def _linear_own(s):
    from block_wise_kv_gb300 import dllm

    case = s["case"]
    if "desc" not in s:  # what a program makes once: the layer's description and the workspace
        act = {"none": dllm.DLLM_ACT_NONE, "silu": dllm.DLLM_ACT_SILU, "gelu": dllm.DLLM_ACT_GELU,
               "gelu_tanh": dllm.DLLM_ACT_GELU_TANH}[case["act"]]
        s["desc"] = dllm.linear_desc(case["k"], case["n"], act, case["gated"], EPS)
        s["ws"] = dllm.workspace(dllm.dllm_linear_workspace_size(s["desc"], case["rows"], case["norm"]))
    dllm.dllm_linear(s["desc"], s["x"], s["w"], s["y"], rms_gain=s["gain"], bias=s["bias"], residual=s["residual"],
                     ws=s["ws"])
    return s["y"]


def _rope_own(s):
    from block_wise_kv_gb300 import dllm

    case = s["case"]
    if "desc" not in s:
        s["desc"] = dllm.layer_desc(case["heads"] * case["d"], case["heads"], case["d"], 5e5, EPS)
    pairs = dllm.DLLM_ROPE_HALVES if case["pairs"] == "halves" else dllm.DLLM_ROPE_NEIGHBOURS
    dllm.dllm_head_norm_rope(s["desc"], s["q"], s["q_out"], s["k"], s["k_out"], s["pos"], s["table"], q_gain=s["q_gain"],
                             k_gain=s["k_gain"], pairs=pairs)
    return {"q": s["q_out"], "k": s["k_out"]}


def _scores_own(s):
    from block_wise_kv_gb300 import dllm

    dllm.dllm_token_scores(s["logits"], s["tokens"], s["logp"], s["lse"], s["entropy"], top_ids=s["top_ids"],
                           top_logp=s["top_logp"], scale=s["case"]["scale"])
    return _scores_outputs(s)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _linear_own, "rope": _rope_own, "scores": _scores_own}[op](state)
    return {"linear": _linear_plain, "rope": _rope_plain, "scores": _scores_plain}[op](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _nearest_bf16(x):
    """float64 -> the nearest value of 8 significant bits, ties to even (of the normal range)."""
    f, e = torch.frexp(x)
    return torch.ldexp(torch.round(f * 256), e - 8)


def _normed(x, gain):
    return x * gain.double() / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS)


def _exact_linear(case, s):
    x = s["x"].double()
    if case["norm"]:
        x = _nearest_bf16(_normed(x, s["gain"]))
    w = s["w"].double()
    t = torch.nn.functional.linear(x, w, None if s["bias"] is None else s["bias"].double())
    g = t.unflatten(-1, (-1, 2))[..., 0] if case["gated"] else t
    if case["act"] == "silu":
        a = g * torch.sigmoid(g)
    elif case["act"] == "gelu":
        a = g * (1 - 0.5 * torch.erfc(g / 2 ** 0.5))
    elif case["act"] == "gelu_tanh":
        a = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    else:
        a = g
    if case["gated"]:
        a = a * t.unflatten(-1, (-1, 2))[..., 1]
    return a if s["residual"] is None else a + s["residual"].double()


def _exact_rope(case, s):
    out = {}
    pos = s["pos"].tolist()
    at = torch.tensor([p for p in pos if p >= 0], device="cuda")
    c, sn = s["table"].double()[at].unbind(-1)
    for name in ("q", "k"):
        x = s[name][:len(at)].double()
        if case["norm"]:
            x = _normed(x, s[name + "_gain"])
        r = case["rotary"]
        i = torch.arange(r // 2, device="cuda")
        first, second = (i, i + r // 2) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(c, sn)[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        full = s[name + "_out"].double()
        full[:len(at)] = y
        out[name] = full
    return out


def _exact_scores(case, s):
    x = s["logits"].double() * case["scale"]
    empty = torch.isneginf(x).all(-1)
    logp = torch.log_softmax(x, -1)
    p = logp.exp()
    out = {"logp": logp.gather(1, s["tokens"].long().clamp(min=0)[:, None])[:, 0], "lse": torch.logsumexp(x, -1),
           "entropy": -torch.special.xlogy(p, p).sum(-1)}
    out["logp"] = torch.where(empty, -math.inf, out["logp"])
    out["logp"] = torch.where(s["tokens"] < 0, 0.0, out["logp"])
    out["entropy"] = torch.where(empty, 0.0, out["entropy"])
    if case["top"]:
        best = torch.where(empty[:, None], -math.inf, logp).topk(case["top"], -1).values
        out["top_ids"], out["top_logp"] = None, best
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "rope": _exact_rope, "scores": _exact_scores}[case["op"]](case, s)
