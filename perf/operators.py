"""Measured calls of the block cache: planning its block tables and slot maps, appending keys and
values to it in 8 bits, and the attention that reads it.

The cache holds K and V as e4m3 codes in blocks of `block` tokens, [blocks, kv heads, block, d], with
one float32 scale for each (block, kv head). A request's block table lists its blocks in order.

  plan     from each request's cached length and number of new tokens: the new tokens' slots
           (block * block size + place in it), their row offsets, the lengths after, and the table
           entries of the blocks that the new tokens open, taken in order from a list of free ones.
  append   the new tokens' K and V (16 bits) into their slots. The scale of a block and head is the
           smallest power of two s with amax / s <= 448 over its tokens' values (at least 2^-40); a
           block that held tokens before keeps the larger of its scale and the new tokens', and its
           codes are brought to it.
  attend   softmax(scale q k^T) v over the cached tokens, for the last q_len tokens of each request
           (causal: query i of a request sees kv_len - q_len + i + 1 keys); query heads share K / V
           heads in groups. A row that sees nothing gives O = 0 and LSE = -inf.
"""
import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_F8 = torch.float8_e4m3fn
_LEAST = -40  # exponent of the smallest scale that append writes


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of a small batch: only latency counts
        dict(name="plan_step_b8", op="plan", B=8, block=64, ctx=4096, new=1, kind="even", shapes=1),
        # one step of a large server: decoding requests and prompts of up to 4096 tokens together
        dict(name="plan_mixed_b4096", op="plan", B=4096, block=128, ctx=16384, new=4096, kind="mixed",
             shapes=2),
        # a decoding step's new tokens, one for each request, into partly filled blocks
        dict(name="append_step_b32_d64", op="append", B=32, H=8, d=64, block=16, dtype="fp16", ctx=2048,
             new=1, kind="step", shapes=3),
        # chunks of a few prompts that end inside blocks
        dict(name="append_ragged_d128", op="append", B=37, H=4, d=128, block=64, dtype="fp16", ctx=4096,
             new=601, kind="ragged", shapes=4),
        # whole prompts (heads and length of the long causal workload)
        dict(name="append_prompt_n16384", op="append", B=2, H=32, d=128, block=128, dtype="bf16", ctx=0,
             new=16384, kind="even", shapes=5),
        # the smallest workload's sizes, one new token
        dict(name="attend_step_b1_h2_n256", op="attend", B=1, H=2, Hkv=2, d=64, block=16, dtype="fp16",
             ctx=256, q=1, kind="even", causal=True, shapes=6),
        # one token for each sequence of the headline workload's shape, a K / V head for each query head
        dict(name="attend_step_b4_h16_n4096", op="attend", B=4, H=16, Hkv=16, d=128, block=128,
             dtype="fp16", ctx=4096, q=1, kind="even", causal=True, shapes=7),
        # two long documents of odd length, four query heads to a K / V head
        dict(name="attend_step_n131071", op="attend", B=2, H=32, Hkv=8, d=128, block=128, dtype="bf16",
             ctx=131071, q=1, kind="even", causal=True, shapes=8),
        # a server's batch: lengths from 0 to 16384
        dict(name="attend_step_ragged_b96", op="attend", B=96, H=32, Hkv=8, d=128, block=64,
             dtype="bf16", ctx=16384, q=1, kind="ragged", causal=True, shapes=9),
        # five drafted tokens for each request, checked in one call
        dict(name="attend_draft_q5_b16", op="attend", B=16, H=32, Hkv=4, d=128, block=32, dtype="fp16",
             ctx=8192, q=5, kind="even", causal=True, shapes=10),
        # prompt chunks of different lengths beside single tokens
        dict(name="attend_chunks_mixed_d64", op="attend", B=9, H=16, Hkv=8, d=64, block=16, dtype="fp16",
             ctx=6000, q=700, kind="mixed", causal=True, shapes=11),
        # the last 2048 tokens of a long prompt (heads and length of the long causal workload)
        dict(name="attend_chunk_q2048_n16384", op="attend", B=1, H=32, Hkv=8, d=128, block=128,
             dtype="bf16", ctx=16384, q=2048, kind="even", causal=True, shapes=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _any(rng)
        w = work(c)
        # no dearer than the largest listed ones, padded to the longest request as the plain form is
        if c["op"] != "attend" or (w["bytes"] <= 1.3e9 and w["flops"] <= 5e11
                                   and c["B"] * c["H"] * c["q"] * c["ctx"] <= 1.07e9
                                   and c["B"] * c["Hkv"] * c["d"] * c["ctx"] <= 1.6e9):
            return c


def _any(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend"])
    c = dict(op=op, block=rng.choice([16, 32, 64, 128]), shapes=rng.randrange(1 << 30))
    if op == "plan":
        B = _log(rng, 1, 4096)
        return dict(c, B=B, ctx=_log(rng, 1, 65536), new=_log(rng, 1, 4096),
                    kind=rng.choice(["even", "step", "ragged", "mixed"]) if B < 256
                    else rng.choice(["step", "mixed"]))
    c.update(d=rng.choice([64, 128]), dtype=rng.choice(["fp16", "bf16"]))
    if op == "append":
        B = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, 32768 // B))
        return dict(c, B=B, H=rng.choice([1, 2, 4, 8, 16, 32]), ctx=_log(rng, 1, 8192) - 1, new=new,
                    kind=rng.choice(["even", "ragged", "mixed"]))
    Hkv = rng.choice([1, 2, 4, 8, 16])
    H = Hkv * rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
    B = _log(rng, 1, 96)
    if rng.random() < 0.6:  # single tokens, or a few
        q = rng.choice([1, 1, 1, 2, 3, 4, 5, 7, 8])
        top = 131072
    else:
        q = _log(rng, 9, 2048)
        top = 16384
    ctx = max(q, _log(rng, 16, top))
    return dict(c, B=B, H=H, Hkv=Hkv, ctx=ctx, q=q, kind=rng.choice(["even", "ragged", "mixed"]),
                causal=rng.random() < 0.85)


def _lengths(c):
    """(cached lengths before, new tokens) of each request for plan and append; (lengths, query
    tokens) for attend. They go by the case alone."""
    r = random.Random(c["shapes"])
    B, ctx, kind = c["B"], c["ctx"], c["kind"]
    most = c["q"] if c["op"] == "attend" else c["new"]
    if kind == "even":
        n, lens = [most] * B, [ctx] * B
    else:
        lens = [r.randint(0, ctx) for _ in range(B)]
        if kind == "step":
            n = [1] * B
        elif kind == "ragged":
            n = [r.randint(1, most) for _ in range(B)]
        else:  # mixed: an eighth of the requests bring many tokens, the others one
            n = [_log(r, 1, most) if i % 8 == 0 else 1 for i in range(B)]
    if c["op"] == "attend" and kind != "even":
        # kept apart from the causal rule: a sequence holds its query tokens, but a free place of the
        # batch has one query token and no keys
        lens = [0 if (m == 1 and r.random() < 0.05) else max(x, m) for x, m in zip(lens, n)]
    return lens, n


def _visible(length, q, causal):
    """Sum over the q query tokens of the keys that each sees."""
    if not causal:
        return q * length
    return sum(max(0, length - q + i + 1) for i in range(q))


def work(case):
    c = case
    lens, n = _lengths(c)
    T, B, bs = sum(n), c["B"], c["block"]
    if c["op"] == "plan":
        opened = sum(-(-(x + m) // bs) - -(-x // bs) for x, m in zip(lens, n))
        return {"bytes": 4.0 * (T + 2 * opened + 2 * B + (B + 1) + B + B), "flops": 0.0}
    if c["op"] == "append":
        blocks = sum(-(-(x + m) // bs) - x // bs for x, m in zip(lens, n) if m)
        return {"bytes": 2.0 * T * c["H"] * c["d"] * (2 + 1) + 4.0 * T + 2 * 4.0 * blocks * c["H"],
                "flops": 2.0 * T * c["H"] * c["d"]}
    blocks = sum(-(-x // bs) for x in lens)
    held = 2.0 * sum(lens) * c["Hkv"] * c["d"] + 2 * 4.0 * blocks * c["Hkv"] + 4.0 * blocks
    rows = T * c["H"]
    pairs = sum(_visible(x, m, c["causal"]) for x, m in zip(lens, n))
    return {"bytes": held + rows * (4.0 * c["d"] + 4) + 8.0 * B, "flops": 4.0 * pairs * c["H"] * c["d"]}


# ------------------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _need(amax):
    """The smallest power of two s with amax / s <= 448, at least 2^-40."""
    m, e = torch.frexp(amax.float())  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, _LEAST)).clamp(min=_LEAST)
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e)


def _held(gen, blocks, heads, bs, d):
    """Codes and scales of filled blocks: normal values, a size of its own for each head."""
    size = torch.exp(0.5 * torch.randn(1, heads, 1, 1, device="cuda", generator=gen))
    x = torch.randn(blocks, heads, bs, d, device="cuda", generator=gen) * size
    s = _need(x.abs().amax(dim=(2, 3)))
    return (x / s[:, :, None, None]).to(_F8), s


def _tables(c, gen, lens, total):
    """Block ids in random order: the blocks held so far in each request's table row (-1 behind
    them), and the others, free."""
    bs = c["block"]
    have = [-(-x // bs) for x in lens]
    width = max(1, max(-(-x // bs) for x in total))
    ids = torch.randperm(sum(-(-x // bs) for x in total) + 3, device="cuda", generator=gen).to(torch.int32)
    col = torch.arange(width, device="cuda")[None]
    hv = torch.tensor(have, device="cuda")
    first = (torch.cumsum(hv, 0) - hv)[:, None]
    inside = col < hv[:, None]
    table = torch.where(inside, ids[(first + col).clamp(max=len(ids) - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), ids[sum(have):].contiguous(), len(ids)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    lens, n = _lengths(c)
    bs = c["block"]
    if c["op"] == "plan":
        table, free, _ = _tables(c, gen, lens, [x + m for x, m in zip(lens, n)])
        # one draw in some runs out of blocks: the last requests that need one are refused
        if c["shapes"] % 4 == 3:
            free = free[: max(1, (3 * len(free)) // 4)].contiguous()
        return dict(op="plan", block=bs, lens=_ints(lens), new=_ints(n), table=table, free=free,
                    pos=_ints([0]), T=sum(n))
    heads = c["H"] if c["op"] == "append" else c["Hkv"]
    total = [x + m for x, m in zip(lens, n)] if c["op"] == "append" else lens
    d, T = c["d"], sum(n)
    table, free, count = _tables(c, gen, total, total)
    k, ks = _held(gen, count, heads, bs, d)
    v, vs = _held(gen, count, heads, bs, d)
    st = dict(op=c["op"], block=bs, k=k, v=v, ks=ks, vs=vs, cache=(k, v, ks, vs))
    if c["op"] == "append":
        start, cnt = torch.tensor(lens, device="cuda"), torch.tensor(n, device="cuda")
        req = torch.repeat_interleave(torch.arange(len(n), device="cuda"), cnt, output_size=T)
        at = torch.arange(T, device="cuda") - (torch.cumsum(cnt, 0) - cnt)[req] + start[req]
        slots = table[req, at // bs] * bs + (at % bs).to(torch.int32)
        size = torch.exp(0.5 * torch.randn(1, heads, 1, device="cuda", generator=gen))
        new = [(torch.randn(T, heads, d, device="cuda", generator=gen) * size).to(_TYPES[c["dtype"]])
               for _ in range(2)]
        return dict(st, kn=new[0], vn=new[1], slots=slots.to(torch.int32).contiguous())
    q = torch.randn(T, c["H"], d, device="cuda", generator=gen).to(_TYPES[c["dtype"]])
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    return dict(st, q=q, table=table, lens=_ints(lens), cu=_ints(cu), causal=c["causal"],
                scale=1.0 / math.sqrt(d), longest=max(lens), most=max(n))


# ------------------------------------------------------------------------------ plain forms

def _plan_plain(s):
    lens, new, bs, T = s["lens"].long(), s["new"].long(), s["block"], s["T"]
    end = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), end])
    have, want = (lens + bs - 1) // bs, (lens + new + bs - 1) // bs
    need = want - have
    upto = s["pos"].long() + torch.cumsum(need, 0)
    granted = (need == 0) | (upto <= len(s["free"]))
    first = upto - need
    kv = lens + torch.where(granted, new, torch.zeros_like(new))
    req = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), new, output_size=T)
    at = torch.arange(T, device="cuda") - cu[req] + lens[req]
    j = at // bs
    fresh = j >= have[req]
    got = s["free"][(first[req] + j - have[req]).clamp(0, len(s["free"]) - 1)].long()
    held = s["table"][req, j.clamp(max=s["table"].shape[1] - 1)].long()
    ids = torch.where(fresh, got, held)
    slots = torch.where(granted[req], ids * bs + at % bs, torch.full_like(at, -1))
    s["table"][req, j] = torch.where(granted[req], ids, held).to(torch.int32)
    used = s["pos"].long() + torch.where(granted, need, torch.zeros_like(need)).sum()
    return slots.to(torch.int32), cu.to(torch.int32), kv.to(torch.int32), s["table"], used.to(torch.int32)


def _store_plain(x, slots, codes, scales, bs):
    """Appends x [T, heads, d] to one of K and V."""
    x = x.float()
    fine = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dim=2)
    blk, off = (slots // bs).long(), (slots % bs).long()
    ids, to = torch.unique(blk, return_inverse=True)
    amax = torch.zeros(len(ids), x.shape[1], device="cuda").index_reduce_(0, to, fine, "amax", include_self=True)
    start = torch.full((len(ids),), bs, device="cuda").index_reduce_(0, to, off, "amin", include_self=True)
    old = scales[ids]
    need = _need(amax)
    now = torch.where(start[:, None] == 0, need, torch.maximum(old, need))
    held = codes.view(torch.uint8)[ids].view(_F8)
    again = (held.float() * (old / now)[:, :, None, None]).to(_F8).view(torch.uint8)
    older = (torch.arange(bs, device="cuda")[None] < start[:, None])[:, None, :, None]
    raw = torch.where(older, again, held.view(torch.uint8))
    raw[to, :, off] = (x / now[to][:, :, None]).to(_F8).view(torch.uint8)
    codes.view(torch.uint8)[ids] = raw
    scales[ids] = now


def _append_plain(s):
    _store_plain(s["kn"], s["slots"], s["k"], s["ks"], s["block"])
    _store_plain(s["vn"], s["slots"], s["v"], s["vs"], s["block"])
    return s["k"], s["v"], s["ks"], s["vs"]


def _rows_plain(codes, scales, table):
    """The cached values [B, heads, keys, d] that a block table lists."""
    B, w = table.shape
    x = codes.view(torch.uint8)[table].view(_F8).float() * scales[table][:, :, :, None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(B, x.shape[2], w * x.shape[3], x.shape[4])


def _attend_plain(s):
    q, lens, cu = s["q"], s["lens"].long(), s["cu"].long()
    T, H, d = q.shape
    B, most = len(lens), s["most"]
    table = s["table"][:, : max(1, -(-s["longest"] // s["block"]))].long().clamp(min=0)
    k, v = _rows_plain(s["k"], s["ks"], table), _rows_plain(s["v"], s["vs"], table)
    heads, keys = k.shape[1], k.shape[2]
    count = cu[1:] - cu[:-1]
    i = torch.arange(most, device="cuda")[None]
    there = i < count[:, None]
    row = (cu[:-1, None] + i).clamp(max=T - 1)
    qq = q[row].float().reshape(B, most, heads, H // heads, d).permute(0, 2, 3, 1, 4)
    x = (qq.reshape(B, heads, -1, d) @ k.transpose(2, 3)) * s["scale"]
    x = x.reshape(B, heads, H // heads, most, keys)
    upto = lens[:, None] - count[:, None] + i + 1 if s["causal"] else lens[:, None].expand(B, most)
    sees = torch.arange(keys, device="cuda") < torch.minimum(upto, lens[:, None])[:, :, None]
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    base = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(x - base)
    total = p.sum(dim=-1, keepdim=True)
    v = torch.where(torch.arange(keys, device="cuda")[:, None] < lens[:, None, None, None], v, torch.zeros((), device="cuda"))
    o = (p.reshape(B, heads, -1, keys) @ v).reshape(B, heads, H // heads, most, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.log(total) + base
    o = o.permute(0, 3, 1, 2, 4).reshape(B, most, H, d)
    lse = lse[..., 0].permute(0, 3, 1, 2).reshape(B, most, H)
    req = torch.repeat_interleave(torch.arange(B, device="cuda"), count, output_size=T)
    at = torch.arange(T, device="cuda") - cu[req]
    return o[req, at].to(q.dtype), lse[req, at]


# ------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        import attention_forward_flashattention_gb300 as fa
        if s["op"] == "plan":
            slots, cu, kv, nxt = fa.cache_plan(s["lens"], s["new"], s["table"], s["free"], s["pos"],
                                               s["T"], s["block"])
            return slots, cu, kv, s["table"], nxt
        if s["op"] == "append":
            fa.cache_append(s["kn"], s["vn"], s["slots"], s["cache"])
            return s["k"], s["v"], s["ks"], s["vs"]
        return fa.attention_forward_cache(s["q"], s["cache"], s["table"], s["lens"], s["cu"],
                                          causal=s["causal"], scale=s["scale"])
    return {"plan": _plan_plain, "append": _append_plain, "attend": _attend_plain}[s["op"]](s)


# ------------------------------------------------------------------------------ 64 bits

def _exact_plan(s):
    lens, new = s["lens"].tolist(), s["new"].tolist()
    table, free, bs = s["table"].tolist(), s["free"].tolist(), s["block"]
    slots, cu, kv, nxt, wanted = [], [0], [], 0, 0
    for b, (x, m) in enumerate(zip(lens, new)):
        need = (x + m + bs - 1) // bs - (x + bs - 1) // bs
        wanted += need
        ok = need == 0 or wanted <= len(free)
        if ok:
            for j in range(need):
                table[b][(x + bs - 1) // bs + j] = free[nxt + j]
            nxt += need
        slots += [table[b][p // bs] * bs + p % bs if ok else -1 for p in range(x, x + m)]
        cu.append(cu[-1] + m)
        kv.append(x + m if ok else x)
    return tuple(_ints(v) for v in (slots, cu, kv, table, [nxt]))


def _exact_store(x, slots, codes, scales, bs):
    """The values before they are rounded to 8 bits, and the scales."""
    x = x.double()
    blocks, heads = scales.shape
    out, old = codes.double(), scales.double()
    blk, off = slots.long() // bs, slots.long() % bs
    place = blk[:, None] * heads + torch.arange(heads, device="cuda")
    big = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    amax = torch.zeros(blocks * heads, dtype=torch.float64, device="cuda")
    amax.scatter_reduce_(0, place.reshape(-1), big.reshape(-1), "amax")
    amax = amax.reshape(blocks, heads)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** (_LEAST + 8)))) - 10  # at or below the wanted exponent
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    need = torch.exp2(e.clamp(min=_LEAST))
    low = torch.full((blocks,), bs, device="cuda").scatter_reduce_(0, blk, off, "amin")
    touched = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    touched[blk] = True
    now = torch.where(low[:, None] == 0, need, torch.maximum(old, need))
    now = torch.where(touched[:, None], now, old)
    held = torch.arange(bs, device="cuda")[None] < torch.where(touched, low, torch.zeros_like(low))[:, None]
    out = torch.where(held[:, None, :, None], out * (old / now)[:, :, None, None], out)
    out[blk, :, off] = x / now[blk][:, :, None]
    return out, now


def _exact_attend(s):
    q, lens, cu, bs = s["q"], s["lens"].tolist(), s["cu"].tolist(), s["block"]
    T, H, d = q.shape
    heads = s["ks"].shape[1]
    g = H // heads
    o = torch.zeros(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        m = cu[b + 1] - cu[b]
        if not length or not m:
            continue
        ids = s["table"][b, : -(-length // bs)].long()
        kk, vv = ((s[t].view(torch.uint8)[ids].view(_F8).double() * s[t + "s"].double()[ids][:, :, None, None])
                  .transpose(0, 1).reshape(heads, -1, d)[:, :length] for t in ("k", "v"))
        for h in range(heads):
            rows = q[cu[b]: cu[b + 1], h * g: (h + 1) * g].double()
            x = torch.einsum("mgd,kd->mgk", rows, kk[h]) * s["scale"]
            if s["causal"]:
                last = length - m + torch.arange(m, device="cuda")
                hidden = torch.arange(length, device="cuda")[None] > last[:, None]
                x = x.masked_fill(hidden[:, None], -math.inf)
            y = torch.logsumexp(x, -1)
            seen = torch.isfinite(y)
            w = torch.where(seen[..., None], torch.exp(x - y[..., None]), 0.0)
            o[cu[b]: cu[b + 1], h * g: (h + 1) * g] = torch.einsum("mgk,kd->mgd", w, vv[h])
            lse[cu[b]: cu[b + 1], h * g: (h + 1) * g] = y
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "plan":
        return _exact_plan(s)
    if s["op"] == "append":
        k, ks = _exact_store(s["kn"], s["slots"], s["k"], s["ks"], s["block"])
        v, vs = _exact_store(s["vn"], s["slots"], s["v"], s["vs"], s["block"])
        return k, v, ks, vs
    return _exact_attend(s)
