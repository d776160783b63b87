"""Plain 64-bit implementations of the 8-bit paged cache's operators, and batches for their tests.

Everything here is written from the definitions in include/dllm.h with torch (float64) or plain Python integers."""
import random

import torch

from block_wise_kv_gb300 import dllm

PAGE = 64
G = 16


def ints(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def cu(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


class Batch:
    """Sequences (n, start, rows) with shuffled pages, as device tensors and a BatchView."""

    def __init__(self, n, start, rows, seed=0, spare=2, cap_rows=None, cap_seq=None, max_block=None, max_seq=None,
                 max_pages=None, first_page=0):
        self.n, self.start, self.rows = list(n), list(start), list(rows)
        pages = [(x + PAGE - 1) // PAGE for x in n]
        self.num_pages = first_page + sum(pages) + spare
        ids = [first_page + i for i in range(sum(pages) + spare)]
        random.Random(seed).shuffle(ids)
        wide = max_pages or max(1, max(pages))
        table = [[-1] * wide for _ in n]
        at = 0
        for b, p in enumerate(pages):
            table[b][:p] = ids[at:at + p]
            at += p
        self.table = table
        self.error = ints([0])
        self.t = dict(table=ints(table), n=ints(n), start=ints(start), rows=ints(rows), cub=ints(cu(rows)), cus=ints(cu(n)))
        self.M = cap_rows if cap_rows is not None else sum(rows)
        self.R = cap_seq if cap_seq is not None else sum(n)
        self.max_block, self.max_seq = max_block or max(1, max(rows)), max_seq or max(1, max(n))
        t = self.t
        self.view = dllm.BatchView(t["table"], t["n"], t["start"], t["rows"], t["cub"], t["cus"], self.M, self.R,
                                   self.max_block, self.max_seq, self.error)

    def bits(self):
        torch.cuda.synchronize()
        return int(self.error.item())


def random_pools(num_pages, kv, d, seed, size=1.0, spread=0.0):
    """Codes drawn as finite e4m3 patterns of normal values, and power-of-two scales."""
    g = torch.Generator("cuda").manual_seed(seed)

    def one():
        x = torch.randn(num_pages, kv, PAGE, d, device="cuda", generator=g) * size
        if spread:
            x = x * torch.exp2((torch.randn(num_pages, kv, PAGE // G, 1, 1, device="cuda", generator=g) * spread).round()).expand(
                -1, -1, -1, G, 1).reshape(num_pages, kv, PAGE, 1)
        grp = x.view(num_pages, kv, PAGE // G, G * d).abs().amax(-1).clamp(min=2.0 ** -50)
        s = torch.exp2(torch.ceil(torch.log2(grp / 448.0)))
        c = (x / s.repeat_interleave(G, 2)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return c, s

    k, ks = one()
    v, vs = one()
    return dllm.Kv8Cache.of(k, v, ks, vs)


def values(codes, scale):
    """The float64 values of whole pools."""
    return codes.view(torch.uint8).view(torch.float8_e4m3fn).float().double() * scale.double().repeat_interleave(G, 2)[..., None]


def attention(b: Batch, q, kv8, scale=None):
    """float64 packed rows: the attention, the log-sum-exp, the attention of |v| (what the rounding of the weights is
    relative to), the largest possible change of a score when q changes by 1, and the largest weight x value scale of
    the row times the sum of |code| (what the weights' smallest step is relative to)."""
    H, d = q.shape[1], q.shape[2]
    kv = kv8.k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.zeros(b.M, H, d, dtype=torch.float64, device="cuda")
    a, lse = torch.zeros_like(o), torch.zeros(b.M, H, dtype=torch.float64, device="cuda")
    small = torch.zeros_like(o)
    reach = torch.zeros(b.M, H, dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, rows) in enumerate(zip(b.n, b.rows)):
        if rows == 0 or n == 0:
            continue
        ids = torch.tensor(b.table[i][:(n + PAGE - 1) // PAGE], device="cuda")
        k, v = (values(c[ids], s[ids]).transpose(0, 1).reshape(kv, -1, d)[:, :n] for c, s in
                ((kv8.k, kv8.k_scale), (kv8.v, kv8.v_scale)))
        rep = H // kv
        k, v = k.repeat_interleave(rep, 0), v.repeat_interleave(rep, 0)
        t = torch.einsum("ihd,hnd->hin", q[at:at + rows].double(), k) * scale
        m = t.amax(-1, keepdim=True)
        p = torch.exp(t - m)
        tot = p.sum(-1, keepdim=True)
        p = p / tot
        o[at:at + rows] = torch.einsum("hin,hnd->ihd", p, v)
        a[at:at + rows] = torch.einsum("hin,hnd->ihd", p, v.abs())
        lse[at:at + rows] = (m + torch.log(tot))[..., 0].T
        vs = kv8.v_scale[ids].double().repeat_interleave(G, 2).transpose(0, 1).reshape(kv, -1)[:, :n].repeat_interleave(rep, 0)
        most = (p * vs[:, None]).amax(-1)  # [H][rows]
        small[at:at + rows] = torch.einsum("hi,hd->ihd", most, (v / vs[..., None]).abs().sum(1))
        reach[at:at + rows] = k.abs().sum(-1).amax(-1)[None] * scale
        at += rows
    return o, lse, a, reach, small


def assert_attention(b, q, kv8, o, lse, scale=None, ref=None):
    """Bounds: the output is rounded to bf16 once (half a step: 2^-8 of the value).  The weights are rounded to 11 bits
    (2^-11 of each, so 2^-11 of the attention of |v|), and as much again covers 2^-22 of each exponential, 32-bit sums
    and a score's error e = 2^-19 max|q| sum|k| (q is held in two 8-bit parts: exact but for what is below 2^-11 of the
    row group's largest, and off by at most 2^-19 of that), which moves a weight by a factor of exp(2 e) at most.
    A weight x value scale is held to an absolute 2^-17 besides (half of the smallest e5m2 step) in units in which the
    row's largest is 2^10 or more: 2^-27 of that largest for each key, times |code|, summed over the keys."""
    o64, lse64, a64, reach, small = ref if ref is not None else attention(b, q, kv8, scale)
    rows = sum(b.rows)
    e = 2.0 ** -19 * q.double().abs().max() * reach[:rows]
    got = o[:rows].double()
    tol = 2.0 ** -8 * o64[:rows].abs() + (2.0 ** -10 + 2 * e)[..., None] * a64[:rows] + 2.0 ** -27 * small[:rows]
    bad = ~((got - o64[:rows]).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float(got[bad][0]), float(o64[:rows][bad][0]))
    if lse is not None:
        off = (lse[:rows].double() - lse64[:rows]).abs()
        ltol = e + 2.0 ** -20 * (1 + lse64[:rows].abs())
        assert (off <= ltol).all(), (float(off.max()), float(ltol.min()))


def e4m3(x):
    """float64 -> the nearest e4m3 value, ties to even, saturated."""
    e = (torch.frexp(x)[1] - 1).clamp(min=-6)
    e = torch.where(x == 0, -6, e)
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def smallest_scale(amax: float) -> float:
    for e in range(-60, 60):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 60


def write(b: Batch, vals, scale, new):
    """The write of rows new [M][kv][d] (float64, finite) into values of codes `vals` (float64 codes) and `scale`, in
    place, group by group."""
    at = 0
    kv = vals.shape[1]
    for i, (n, s, rows) in enumerate(zip(b.n, b.start, b.rows)):
        for g in range(s // G, (s + rows + G - 1) // G if rows else s // G):
            page, quarter = b.table[i][g * G // PAGE], g % (PAGE // G)
            slots = [(p, p % PAGE) for p in range(g * G, g * G + G) if p < n]
            fresh = [(p, t) for p, t in slots if s <= p < s + rows]
            kept = [t for p, t in slots if not s <= p < s + rows]
            for h in range(kv):
                x = torch.stack([new[at + p - s, h] for p, _ in fresh])
                want = smallest_scale(float(x.abs().max()))
                old = float(scale[page, h, quarter])
                if kept:
                    want = max(want, old)
                    vals[page, h, kept] = e4m3(vals[page, h, kept] * (old / want))
                scale[page, h, quarter] = want
                vals[page, h, [t for _, t in fresh]] = e4m3(x / want)
        at += rows


def plan(n, start, rows, held, table, ring, state, cap):
    """The batch plan in plain integers; table and ring are changed in place."""
    P = len(ring)
    head, count = state
    need = [(x + PAGE - 1) // PAGE for x in n]
    asked = given = granted = 0
    now, short = [], False
    fresh = {}
    back = []
    for b, (nd, h) in enumerate(zip(need, held)):
        if nd > h:
            asked += nd - h
            if asked > count:
                now.append(h)
                short = True
                continue
            for k in range(nd - h):
                fresh[(b, h + k)] = ring[(head + asked - (nd - h) + k) % P]
            granted = asked
        elif nd < h:
            back += table[b][nd:h]
        now.append(nd)
    given = len(back)
    for (b, p), i in fresh.items():
        table[b][p] = i
    for k, i in enumerate(back):
        ring[(head + count + k) % P] = i
    slot, seq, pos = [], [], []
    for b in range(len(n)):
        for i in range(rows[b]):
            p = start[b] + i
            seq.append(b)
            pos.append(p)
            slot.append(table[b][p // PAGE] * PAGE + p % PAGE if p // PAGE < now[b] else -1)
    fill = [-1] * (cap - len(slot))
    return now, [(head + granted) % P, count - granted + given], cu(rows), cu(n), slot + fill, seq + fill, pos + fill, short
