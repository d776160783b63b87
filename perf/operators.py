"""Cases, inputs, plain forms and 64-bit forms of the 8-bit paged cache's operators.

Three operators that a server runs one after the other:

* ``plan``: the batch made on the GPU from request lengths: pages taken from and given back to a ring of free
  pages, block table, prefix sums, and for each block row its sequence, position and cache slot
  (``dllm_batch_plan``);
* ``write``: rows of K and V quantised to e4m3 into the paged cache, a power-of-two scale for each 16 tokens of a
  head, from packed rows (``dllm_kv8_write``) or from the bf16 pools (``dllm_kv8_write_pool``);
* ``attend``: the attention of the block rows over that cache, grouped heads, with the log-sum-exp
  (``dllm_kv8_attention``).

Where ``own`` is false, ``run`` computes them with elementary torch operations in 32 bits; where it is true it makes the
library's calls.
"""
import math
import random

import torch

own = False

PAGE = 64
GROUP = 16
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The smallest call of the attention: the repository's tiny workload (4 heads of 64, 320 tokens, a block of 32).
        dict(name="attend_tiny", op="attend", batch=1, len_lo=320, len_hi=320, rows_lo=32, rows_hi=32, heads=4,
             kv_heads=4, d=64, shape=1),
        # One sequence of the LLaDA-shaped layer: the latency of a single user's inner step.
        dict(name="attend_single", op="attend", batch=1, len_lo=768, len_hi=768, rows_lo=32, rows_hi=32, heads=32,
             kv_heads=32, d=128, shape=2),
        # The repository's headline batch: 16 sequences of 1536 tokens, blocks of 32.
        dict(name="attend_stack", op="attend", batch=16, len_lo=1536, len_hi=1536, rows_lo=32, rows_hi=32, heads=32,
             kv_heads=32, d=128, shape=3),
        # A mixed batch in mid-service: the ragged workload's lengths, odd block lengths among them.
        dict(name="attend_ragged", op="attend", batch=32, len_lo=128, len_hi=4608, rows_lo=16, rows_hi=64, heads=32,
             kv_heads=32, d=128, shape=4),
        # Single-token decoding with grouped heads, lengths from one token to long ones.
        dict(name="attend_token_gqa", op="attend", batch=64, len_lo=1, len_hi=16384, rows_lo=1, rows_hi=1, heads=32,
             kv_heads=8, d=128, shape=5),
        # Two very long contexts, a few rows each: one sequence's keys have to be spread over the whole GPU.
        dict(name="attend_long_gqa", op="attend", batch=2, len_lo=98317, len_hi=131072, rows_lo=4, rows_hi=4, heads=32,
             kv_heads=8, d=128, shape=6),
        # Blocks of 32 with four query heads to each key head: 128 rows on every key.
        dict(name="attend_block_gqa", op="attend", batch=8, len_lo=1000, len_hi=8192, rows_lo=32, rows_hi=32, heads=32,
             kv_heads=8, d=128, shape=7),
        # One new token of each sequence appended: mostly groups that hold earlier tokens already.
        dict(name="write_token_gqa", op="write", source="rows", batch=128, len_lo=1, len_hi=8192, rows_lo=1, rows_hi=1,
             kv_heads=8, d=128, shape=8),
        # The inner step's write: the blocks of the headline batch.
        dict(name="write_block", op="write", source="rows", batch=16, len_lo=1500, len_hi=1536, rows_lo=32, rows_hi=32,
             kv_heads=32, d=128, shape=9),
        # A block boundary: whole sequences of the long workload out of the bf16 pools.
        dict(name="write_pool_boundary", op="write", source="pool", batch=4, len_lo=5120, len_hi=5120, rows_lo=0,
             rows_hi=0, kv_heads=32, d=128, shape=10),
        # A step of a running batch: sequences grow by a block, some end, some begin.
        dict(name="plan_step", op="plan", mode="step", batch=64, len_lo=128, len_hi=4608, rows=32, free=2.0, shape=11),
        # Admission of many prompts at once: every row of every prompt gets its slot.
        dict(name="plan_prompts", op="plan", mode="prompts", batch=512, len_lo=1, len_hi=8192, rows=0, free=1.5,
             shape=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "plan"])
    shape = rng.randrange(1 << 30)
    if op == "plan":
        mode = rng.choice(["step", "prompts"])
        batch = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, 8192)
        return dict(op=op, mode=mode, batch=batch, len_lo=_log_int(rng, 1, hi), len_hi=hi,
                    rows=rng.randint(1, 64) if mode == "step" else 0, free=rng.choice([0.6, 1.0, 3.0]), shape=shape)
    d = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8, 16, 32]) * (128 // d)
    if op == "write":
        source = rng.choice(["rows", "pool"])
        batch = _log_int(rng, 1, 128)
        most = max(1, min(8192, 4 * 5120 * 32 * 128 // (batch * kv * d)))
        hi = _log_int(rng, 1, most)
        whole = rng.random() < 0.3
        lo_rows = 0 if whole else rng.randint(1, 64)
        return dict(op=op, source=source, batch=batch, len_lo=_log_int(rng, 1, hi), len_hi=hi, rows_lo=lo_rows,
                    rows_hi=0 if whole else rng.randint(lo_rows, 64), kv_heads=kv, d=d, shape=shape)
    group = rng.choice([1, 1, 2, 4, 8])
    batch = _log_int(rng, 1, 64)
    rows_hi = _log_int(rng, 1, 64)
    most = max(1, min(131072, 32 * 4608 * 32 * 128 // (batch * kv * d), 32 * 32 * 64 * 4608 // (batch * kv * group * rows_hi)))
    hi = _log_int(rng, 1, most)
    return dict(op=op, batch=batch, len_lo=_log_int(rng, 1, hi), len_hi=hi, rows_lo=rng.randint(1, rows_hi),
                rows_hi=rows_hi, heads=kv * group, kv_heads=kv, d=d, shape=shape)


def _lengths(case):
    """Lengths, first rows and row counts of the blocks, the same for every seed."""
    r = random.Random(case["shape"])
    n = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    if case["op"] == "plan":
        if case["mode"] == "prompts":
            return n, [0] * len(n), list(n), [0] * len(n)
        held = [(x + PAGE - 1) // PAGE for x in n]
        rows = [case["rows"]] * len(n)
        n = [x + case["rows"] for x in n]
        for b in range(len(n)):
            what = r.random()
            if what < 0.1:  # has ended: its pages go back
                n[b], rows[b] = 0, 0
            elif what < 0.2:  # has just come: it has none yet
                held[b] = 0
        return n, [x - k for x, k in zip(n, rows)], rows, held
    if case["rows_hi"] == 0:
        return n, [0] * len(n), list(n), None
    rows = [min(x, r.randint(case["rows_lo"], case["rows_hi"])) for x in n]
    if case["op"] == "write" and case["rows_hi"] == 1:
        return n, [x - 1 for x in n], rows, None
    return n, [r.randint(0, x - k) for x, k in zip(n, rows)], rows, None


def work(case):
    n, _, rows, held = _lengths(case)
    pages = [(x + PAGE - 1) // PAGE for x in n]
    if case["op"] == "plan":
        moved = sum(abs(p - h) for p, h in zip(pages, held))
        return {"bytes": 16 * len(n) + 8 * moved + 12 * len(n) + 12 * sum(rows), "flops": 0}
    hd = case["kv_heads"] * case["d"]
    if case["op"] == "write":
        groups = sum((k + GROUP - 1) // GROUP for k in rows)
        return {"bytes": sum(rows) * hd * 2 * 3 + groups * case["kv_heads"] * 8, "flops": 0}
    kv = sum(n) * hd * 2 + sum((x + GROUP - 1) // GROUP for x in n) * case["kv_heads"] * 8
    qo = sum(rows) * case["heads"] * (case["d"] * 4 + 4)
    return {"bytes": kv + qo, "flops": 4 * case["heads"] * case["d"] * sum(x * k for x, k in zip(n, rows))}


# ------------------------------------------------------------------ inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


def _power_of_two(amax):
    """The smallest power of two that brings amax within 448, at least 2^-60 and at most 2^60."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(torch.int32)  # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp(-60, 60)
    return ((e + 127) << 23).view(torch.float32)


def _codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _filled_pool(pages, kv, d, gen, spread):
    """A pool of codes and scales of normally distributed rows whose columns have different sizes."""
    column = torch.exp(spread * torch.randn(kv, 1, d, device="cuda", generator=gen))
    codes = torch.empty(pages, kv, PAGE, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(pages, kv, PAGE // GROUP, device="cuda")
    step = max(1, (1 << 28) // (kv * PAGE * d))
    for p in range(0, pages, step):
        x = torch.randn(min(step, pages - p), kv, PAGE, d, device="cuda", generator=gen) * column
        s = _power_of_two(x.view(x.shape[0], kv, PAGE // GROUP, -1).abs().amax(-1))
        scale[p:p + step] = s
        codes[p:p + step] = _codes(x / s.repeat_interleave(GROUP, 2).unsqueeze(-1))
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    n, start, rows, held = _lengths(case)
    pages = [(x + PAGE - 1) // PAGE for x in n]
    s = dict(case=case, seq_len=_ints(n), block_start=_ints(start), block_len=_ints(rows))
    batch = len(n)
    if case["op"] == "plan":
        wide = max(1, max(pages), max(held))
        asked = sum(max(0, p - h) for p, h in zip(pages, held))
        free = int(asked * case["free"]) + 1
        total = sum(held) + free + PAGE  # as many pages more are in other hands
        ids = torch.randperm(total, device="cuda", generator=gen, dtype=torch.int32)
        table = torch.full((batch, wide), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(wide, device="cuda")
        table[col[None] < _ints(held)[:, None]] = ids[:sum(held)]
        head = random.Random(seed).randrange(total)
        ring = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(free, device="cuda")) % total] = ids[sum(held):sum(held) + free]
        cap = sum(rows) + batch
        s.update(held=_ints(held), table=table, ring=ring, ring_state=_ints([head, free]), ring_next=_ints([0, 0]),
                 held_next=_ints([0] * batch), cu_block=_ints([0] * (batch + 1)), cu_seq=_ints([0] * (batch + 1)),
                 row_slot=_ints([0]).expand(cap).clone(), row_seq=_ints([0]).expand(cap).clone(),
                 row_pos=_ints([0]).expand(cap).clone(), cap=cap, most_rows=max(1, max(rows)), most=max(1, max(n)),
                 sum_rows=cap, sum_seq=sum(n))
        return s
    kv, d = case["kv_heads"], case["d"]
    total = sum(pages) + 3
    ids = torch.randperm(total, device="cuda", generator=gen, dtype=torch.int32)
    table = torch.zeros(batch, max(pages), dtype=torch.int32, device="cuda")
    col = torch.arange(max(pages), device="cuda")
    table[col[None] < _ints(pages)[:, None]] = ids[:sum(pages)]
    k_codes, k_scale = _filled_pool(total, kv, d, gen, 0.5)
    v_codes, v_scale = _filled_pool(total, kv, d, gen, 0.3)
    s.update(table=table, k=k_codes, v=v_codes, k_scale=k_scale, v_scale=v_scale, cu_block=_ints(_cu(rows)),
             cu_seq=_ints(_cu(n)), sum_rows=sum(rows), sum_seq=sum(n), most_rows=max(rows), most=max(n), pages=total)
    if case["op"] == "attend":
        # What lies behind the end of a sequence in its last page is never attended to: not-a-number codes and scales.
        last = s["table"].gather(1, ((s["seq_len"] - 1) // PAGE).long()[:, None])[:, 0].long()
        slot = torch.arange(PAGE, device="cuda")
        used = (s["seq_len"] - 1) % PAGE + 1
        for pool, scale in ((k_codes, k_scale), (v_codes, v_scale)):
            tail = pool.view(torch.uint8)[last]
            tail.masked_fill_((slot[None] >= used[:, None])[:, None, :, None], 0x7F)
            pool.view(torch.uint8)[last] = tail
            over = scale[last]
            over.masked_fill_((slot[::GROUP][None] >= used[:, None])[:, None, :], float("nan"))
            scale[last] = over
        s["q"] = torch.randn(sum(rows), case["heads"], d, device="cuda", generator=gen).to(torch.bfloat16)
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(sum(rows), case["heads"], device="cuda")
        return s
    shape = (sum(rows), kv, d) if case["source"] == "rows" else (total, kv, PAGE, d)
    size = torch.exp(0.5 * torch.randn(kv, 1, d, device="cuda", generator=gen))
    for name in ("k_new", "v_new"):
        x = torch.randn(shape, device="cuda", generator=gen)
        s[name] = (x * (size[:, 0] if case["source"] == "rows" else size)).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ the plain forms
def _rows_of(s, cap, cu):
    """Sequence, position and validity of each packed block row."""
    j = torch.arange(cap, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu[1:], j, right=True).clamp(max=s["seq_len"].numel() - 1)
    return b, s["block_start"][b] + j - cu[b], j < cu[-1]


def _plan_plain(s):
    n, held, table, ring = s["seq_len"], s["held"], s["table"], s["ring"]
    total = ring.numel()
    head, free = s["ring_state"][0], s["ring_state"][1]
    need = (n + PAGE - 1) // PAGE
    take, give = (need - held).clamp(min=0), (held - need).clamp(min=0)
    take_to, give_to = torch.cumsum(take, 0), torch.cumsum(give, 0)
    granted = (take_to <= free) & (take > 0)
    held_next = torch.where((take > 0) & ~granted, held, need)
    taken = torch.where(granted, take, 0).sum()
    col = torch.arange(table.shape[1], device="cuda")[None]
    fresh = granted[:, None] & (col >= held[:, None]) & (col < need[:, None])
    source = (head + (take_to - take)[:, None] + col - held[:, None]) % total
    back = (col >= need[:, None]) & (col < held[:, None])
    to = torch.where(back, (head + free + (give_to - give)[:, None] + col - need[:, None]) % total, total)
    longer = torch.cat([ring, ring[:1]])
    longer.scatter_(0, to.reshape(-1), table.reshape(-1))
    table.copy_(torch.where(fresh, ring[source], table))
    ring.copy_(longer[:total])
    s["held_next"].copy_(held_next)
    s["ring_next"].copy_(torch.stack([(head + taken) % total, free - taken + give_to[-1]]))
    s["cu_block"][1:] = torch.cumsum(s["block_len"], 0)
    s["cu_seq"][1:] = torch.cumsum(n, 0)
    b, pos, there = _rows_of(s, s["cap"], s["cu_block"])
    page = table[b, (pos // PAGE).clamp(0, table.shape[1] - 1)]
    s["row_slot"].copy_(torch.where(there & (pos // PAGE < held_next[b]), page * PAGE + pos % PAGE, -1))
    s["row_seq"].copy_(torch.where(there, b, -1))
    s["row_pos"].copy_(torch.where(there, pos, -1))
    return _plan_outputs(s)


def _plan_outputs(s):
    return {k: s[k] for k in ("table", "ring", "held_next", "ring_next", "cu_block", "cu_seq", "row_slot", "row_seq",
                              "row_pos")}


def _quantise_plain(s, pool, scale, new, b, pos):
    """The rows `new` into one pool: scales of the touched groups, the kept rows of the first and last group of each
    block in the new scale, then the rows."""
    kv = pool.shape[1]
    page = s["table"][b, pos // PAGE].long()
    slot = (pos % PAGE).long()
    if s["case"]["source"] == "pool":
        new = new[page, :, slot]
    x = new.float()
    amax = x.abs().amax(-1)
    group = page * (PAGE // GROUP) + slot // GROUP
    most = torch.zeros(pool.shape[0] * (PAGE // GROUP), kv, device="cuda")
    most.scatter_reduce_(0, group[:, None].expand(-1, kv), amax, "amax")
    first, end = s["block_start"], s["block_start"] + s["block_len"]
    edge = torch.stack([first // GROUP, (end - 1) // GROUP], 1)  # [batch][2]
    epage = s["table"].gather(1, (edge * GROUP // PAGE).long()).long()
    egroup = edge.long() % (PAGE // GROUP)
    epos = edge[:, :, None] * GROUP + torch.arange(GROUP, device="cuda")
    kept = (epos < s["seq_len"][:, None, None]) & ((epos < first[:, None, None]) | (epos >= end[:, None, None]))
    old = scale[epage, :, egroup]  # [batch][2][kv]
    need = _power_of_two(most[epage * (PAGE // GROUP) + egroup])
    wanted = torch.where(kept.any(-1)[..., None], torch.maximum(old, need), need)
    scale[page, :, slot // GROUP] = _power_of_two(most[group])
    scale[epage, :, egroup] = wanted
    eslot = (epos % PAGE).long()
    bits = pool.view(torch.uint8)
    there = bits[epage[..., None], :, eslot]  # [batch][2][16][kv][d]
    again = _codes(there.view(torch.float8_e4m3fn).float() * (old / wanted)[:, :, None, :, None]).view(torch.uint8)
    bits[epage[..., None], :, eslot] = torch.where(kept[..., None, None], again, there)
    bits[page, :, slot] = _codes(x / scale[page, :, slot // GROUP][..., None]).view(torch.uint8)


def _write_plain(s):
    b, pos, _ = _rows_of(s, s["sum_rows"], s["cu_block"])
    _quantise_plain(s, s["k"], s["k_scale"], s["k_new"], b, pos)
    _quantise_plain(s, s["v"], s["v_scale"], s["v_new"], b, pos)
    return _write_outputs(s)


def _write_outputs(s):
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale")}


def _gathered(s, pool, scale, there):
    """[batch][kv][most][d] of a pool's values in 32 bits, zero behind the end of a sequence."""
    page = s["table"].long()
    x = pool.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()  # [batch][pages][kv][64][d]
    x = x * scale[page].repeat_interleave(GROUP, 3)[..., None]
    x = x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, x.shape[4])
    return torch.where(there[:, None, :, None], x, 0.0)


def _attend_plain(s):
    case = s["case"]
    heads, kv, d, batch = case["heads"], case["kv_heads"], case["d"], case["batch"]
    there = torch.arange(s["table"].shape[1] * PAGE, device="cuda")[None] < s["seq_len"][:, None]
    b, pos, _ = _rows_of(s, s["sum_rows"], s["cu_block"])
    i = pos - s["block_start"][b]
    q = torch.zeros(batch, s["most_rows"], heads, d, device="cuda")
    q[b, i] = s["q"].float() * (1.0 / math.sqrt(d))
    q = q.view(batch, s["most_rows"], kv, heads // kv, d).permute(0, 2, 1, 3, 4).reshape(batch, kv, -1, d)
    t = q @ _gathered(s, s["k"], s["k_scale"], there).transpose(2, 3)
    t = t.masked_fill_(~there[:, None, None], float("-inf"))
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = (p @ _gathered(s, s["v"], s["v_scale"], there)) / total
    back = lambda x: x.view(batch, kv, s["most_rows"], heads // kv, -1).permute(0, 2, 1, 3, 4).reshape(batch, s["most_rows"], heads, -1)[b, i]  # noqa: E731
    s["o"].copy_(back(o))
    s["lse"].copy_(back(m + torch.log(total))[..., 0])
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ the library's calls
def _handle(s):
    """The structs and the workspace that a program keeps from one call to the next."""
    from block_wise_kv_gb300 import dllm

    if "handle" in s:
        return dllm, s["handle"]
    case = s["case"]
    view = dllm.BatchView(s["table"], s["seq_len"], s["block_start"], s["block_len"], s["cu_block"], s["cu_seq"],
                          s["sum_rows"], s["sum_seq"], s["most_rows"], s["most"])
    h = {"batch": view}
    if case["op"] == "plan":
        h["ring"] = dllm.PageRing(s["ring"], s["ring_state"], s["ring_next"])
    else:
        heads = case.get("heads", case["kv_heads"])
        h["desc"] = dllm.layer_desc(heads * case["d"], heads, case["d"], 10000.0)
        h["kv8"] = dllm.Kv8Cache.of(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "attend":
        h["ws"] = dllm.workspace(dllm.dllm_kv8_attention_workspace_size(h["desc"], view.c, h["kv8"].c))
    if case.get("source") == "pool":
        h["cache"] = dllm.CacheC(s["k_new"].data_ptr(), s["v_new"].data_ptr(), None, None, None, None, s["pages"], None,
                                 None, None)
    s["handle"] = h
    return dllm, h


def _plan_own(s):
    dllm, h = _handle(s)
    dllm.dllm_batch_plan(h["batch"].c, s["held"], s["held_next"], s["table"], s["cu_block"], s["cu_seq"], h["ring"].c,
                         s["row_slot"], s["row_seq"], s["row_pos"])
    return _plan_outputs(s)


def _write_own(s):
    dllm, h = _handle(s)
    if s["case"]["source"] == "rows":
        dllm.dllm_kv8_write(h["desc"], h["batch"].c, s["k_new"], s["v_new"], h["kv8"].c)
    else:
        dllm.dllm_kv8_write_pool(h["desc"], h["batch"].c, h["cache"], h["kv8"].c)
    return _write_outputs(s)


def _attend_own(s):
    dllm, h = _handle(s)
    dllm.dllm_kv8_attention(h["desc"], h["batch"].c, s["q"], h["kv8"].c, s["o"], s["lse"], h["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _plan_own, "write": _write_own, "attend": _attend_own}[op](state)
    return {"plan": _plan_plain, "write": _write_plain, "attend": _attend_plain}[op](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _two_to(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_exact(x):
    """float64 -> the nearest e4m3 value (ties to even), for |x| <= 448."""
    e = (torch.frexp(x)[1] - 1).clamp(min=-6)
    e = torch.where(x == 0, -6, e)
    step = _two_to(e - 3)
    return torch.round(x / step) * step


def _scale_exact(amax):
    """The power of two 2^e, -60 <= e <= 60, of the smallest e with 448 2^e >= amax."""
    best = _two_to(torch.full(amax.shape, 60, device=amax.device))
    for e in range(59, -61, -1):
        best = torch.where(amax <= E4M3_MAX * 2.0 ** e, 2.0 ** e, best)
    return best


def _exact_attend(case, s):
    n, _, rows, _ = _lengths(case)
    group, d = case["heads"] // case["kv_heads"], case["d"]
    out, lse, at = [], [], 0
    for b, (length, k) in enumerate(zip(n, rows)):
        ids = s["table"][b, :(length + PAGE - 1) // PAGE].long()
        full = []
        for pool, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            x = pool.view(torch.uint8)[ids].view(torch.float8_e4m3fn).to(torch.float32).double()
            x = x.view(*x.shape[:2], PAGE // GROUP, GROUP, d) * scale[ids].double()[..., None, None]
            full.append(x.view(len(ids), -1, PAGE, d).transpose(0, 1).reshape(case["kv_heads"], -1, d)[:, :length])
        q = s["q"][at:at + k].double().transpose(0, 1).reshape(case["kv_heads"], group * k, d)
        t = torch.matmul(q, full[0].transpose(1, 2)) * (d ** -0.5)
        norm = torch.logsumexp(t, -1, keepdim=True)
        o = torch.matmul(torch.exp(t - norm), full[1])
        out.append(o.reshape(case["heads"], k, d).transpose(0, 1))
        lse.append(norm.reshape(case["heads"], k).transpose(0, 1))
        at += k
    return {"o": torch.cat(out), "lse": torch.cat(lse)}


def _exact_write(case, s):
    n, start, rows, _ = _lengths(case)
    table = s["table"].cpu()
    out = {}
    for what in ("k", "v"):
        codes = s[what].view(torch.uint8).view(torch.float8_e4m3fn).to(torch.float32).double()
        scale, new = s[what + "_scale"].double().clone(), s[what + "_new"]
        at = 0
        for b in range(len(n)):
            lo, hi = start[b], start[b] + rows[b]
            for p0 in range(lo // PAGE * PAGE, hi, PAGE):  # page by page
                page = int(table[b, p0 // PAGE])
                g0, g1 = max(0, lo - p0) // GROUP, (min(PAGE, hi - p0) + GROUP - 1) // GROUP
                pos = p0 + g0 * GROUP + torch.arange((g1 - g0) * GROUP, device="cuda")
                fresh = (pos >= lo) & (pos < hi)
                keep = (pos < n[b]) & ~fresh
                if case["source"] == "rows":
                    x = new[at + (pos - lo).clamp(0, rows[b] - 1)].double().transpose(0, 1)
                else:
                    x = new[page, :, g0 * GROUP:g1 * GROUP].double()
                x = torch.where(fresh[None, :, None], x, 0.0).unflatten(1, (g1 - g0, GROUP))
                amax = x.abs().amax((2, 3))
                need = _scale_exact(amax)
                old = scale[page, :, g0:g1]
                has = keep.view(g1 - g0, GROUP).any(-1)
                now = torch.where(has[None], torch.maximum(old, need), need)
                c = codes[page, :, g0 * GROUP:g1 * GROUP].unflatten(1, (g1 - g0, GROUP))
                kept = _e4m3_exact(c * (old / now)[..., None, None])
                mine = torch.where(fresh.view(1, -1, GROUP, 1), _e4m3_exact(x / now[..., None, None]),
                                   torch.where(keep.view(1, -1, GROUP, 1), kept, c))
                codes[page, :, g0 * GROUP:g1 * GROUP] = mine.flatten(1, 2)
                scale[page, :, g0:g1] = now
            at += rows[b]
        out[what], out[what + "_scale"] = codes, scale
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return _exact_attend(case, s) if case["op"] == "attend" else _exact_write(case, s)
