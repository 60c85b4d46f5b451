"""Measured calls around attention: queries and keys normalised and rotated before it, a tree of drafted
tokens attending over the block cache, and what happens to the cache's blocks afterwards.

  rope     RMS norm of every head of q and k with learned weights, then rotation by the tokens'
           positions (cos and sin from a table), in one pass; and its gradients.
  attend   from the drafted tokens' parents: which of them each one sees (itself and its ancestors, as
           bits) and its position; then softmax(scale q k^T) v of the drafted tokens over their context
           and the drafted tokens that they see, from the 8-bit block cache. The drafted tokens are the
           sequence's last ones; query heads share K / V heads in groups. A row that sees nothing gives
           O = 0 and LSE = -inf.
  keep     after the drafts have been judged: the kept ones of each request move together behind its
           context, in the cache, and the blocks that this leaves empty go back to the free list. A
           block into which tokens move takes the largest scale of what it then holds.
  fork     requests that go on from another one's tokens (samples of one prompt, a beam): they share its
           full blocks, whose counts go up, and get a copy of the last one.
"""
import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_F8 = torch.float8_e4m3fn
_LEAST = -40  # exponent of the smallest scale


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token for each sequence of the headline workload's shape: only latency counts
        dict(name="rope_step_b4_h16", op="rope", B=1, N=4, H=16, Hkv=16, d=128, dtype="fp16", r=128,
             pairs=False, weights="same", grad=False, layout="fused", top=4096),
        # a prompt of the long causal workload's length, from a fused projection's rows
        dict(name="rope_prompt_n16384", op="rope", B=1, N=16384, H=32, Hkv=8, d=128, dtype="bf16", r=128,
             pairs=False, weights="same", grad=False, layout="fused", top=16384),
        # a training step (forward and backward) of the headline workload's shape
        dict(name="rope_train_b4_h16_n4096", op="rope", B=4, N=4096, H=16, Hkv=16, d=128, dtype="fp16",
             r=128, pairs=False, weights="fp32", grad=True, layout="heads", top=4096),
        # one of the small-head-dimension workload's, neighbouring elements as pairs, half of them turned
        dict(name="rope_train_b2_h32_n8191_d64", op="rope", B=2, N=8191, H=32, Hkv=4, d=64, dtype="bf16",
             r=32, pairs=True, weights="same", grad=True, layout="tokens", top=8192),
        # the smallest workload's sizes, five drafted tokens
        dict(name="attend_tree_b1_h2_n256", op="attend", B=1, H=2, Hkv=2, d=64, block=16, dtype="fp16",
             ctx=256, q=5, kind="even", flat=False, shapes=1),
        # drafts of 13 tokens for each request of a server's batch
        dict(name="attend_tree_b16_n8192", op="attend", B=16, H=32, Hkv=4, d=128, block=32, dtype="fp16",
             ctx=8192, q=13, kind="even", flat=False, shapes=2),
        # trees of up to 64 tokens, contexts of 0 to 16384
        dict(name="attend_tree_ragged_b32", op="attend", B=32, H=32, Hkv=8, d=128, block=64, dtype="bf16",
             ctx=16384, q=64, kind="ragged", flat=True, shapes=3),
        # two long documents of odd length, four drafted tokens each
        dict(name="attend_tree_n131071", op="attend", B=2, H=32, Hkv=8, d=128, block=128, dtype="bf16",
             ctx=131071, q=4, kind="even", flat=True, shapes=4),
        # a step of a small batch: a path of a few tokens, one or two blocks each
        dict(name="keep_b16_h4", op="keep", B=16, H=4, d=128, block=32, ctx=2048, n=13, kind="path",
             shapes=5),
        # a large batch: any half of 96 tokens stays
        dict(name="keep_b256_h32", op="keep", B=256, H=32, d=128, block=128, ctx=512, n=96, kind="any",
             shapes=6),
        # four samples of one prompt of odd length
        dict(name="fork_b4_n4095", op="fork", B=1, n=4, H=8, d=64, block=64, ctx=4095, kind="even",
             shapes=7),
        # a beam of 8 for each of 64 requests
        dict(name="fork_beam_b64_n8", op="fork", B=64, n=512, H=32, d=128, block=128, ctx=512,
             kind="ragged", shapes=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _any(rng)
        w = work(c)
        if c["op"] == "attend":
            # no dearer than the largest listed ones, padded to the longest request as the plain form is
            if (w["bytes"] <= 1.2e9 and w["flops"] <= 3e11 and c["B"] * c["H"] * c["q"] * c["ctx"] <= 1.07e9
                    and c["B"] * c["Hkv"] * c["d"] * (c["ctx"] + c["q"]) <= 1.1e9):
                return c
        elif w["bytes"] <= (1.3e9 if c["op"] == "rope" else 4e8) and _held_bytes(c) <= 3e9:
            return c


def _held_bytes(c):
    return 0 if c["op"] == "rope" else 2.0 * c["B"] * (c["ctx"] + c["n"] + c["block"]) * c["H"] * c["d"]


def _any(rng):
    op = rng.choice(["rope", "rope", "attend", "attend", "attend", "keep", "fork"])
    d = rng.choice([64, 128])
    if op == "rope":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        grad = rng.random() < 0.5
        B = rng.choice([1, 2, 3, 4]) if grad else 1
        return dict(op=op, B=B, N=_log(rng, 1, 32768), H=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv, d=d,
                    dtype=rng.choice(["fp16", "bf16"]), r=rng.choice([d, d, d // 2, 16]),
                    pairs=rng.random() < 0.4, weights=rng.choice(["same", "fp32", "none"]), grad=grad,
                    layout=rng.choice(["fused", "heads", "tokens"]), top=_log(rng, 16, 131072))
    c = dict(op=op, d=d, block=rng.choice([16, 32, 64, 128]), shapes=rng.randrange(1 << 30))
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        q = _log(rng, 1, 96)
        kind = rng.choice(["even", "ragged", "ragged"])
        return dict(c, B=_log(rng, 1, 96), H=Hkv * rng.choice([1, 1, 2, 3, 4, 6, 8]), Hkv=Hkv, q=q,
                    ctx=_log(rng, 1, 131072 if q <= 8 else 16384), dtype=rng.choice(["fp16", "bf16"]),
                    kind=kind, flat=kind == "ragged" or rng.random() < 0.5)
    H = rng.choice([1, 2, 4, 8, 16, 32])
    if op == "keep":
        return dict(c, B=_log(rng, 1, 256), H=H, ctx=_log(rng, 1, 4096), n=_log(rng, 1, 96),
                    kind=rng.choice(["path", "path", "any"]))
    B = _log(rng, 1, 64)
    return dict(c, B=B, n=B * rng.randint(1, 8), H=H, ctx=_log(rng, 1, 8192),
                kind=rng.choice(["even", "ragged"]))


def _words(c):
    """64-bit words that hold a bit for each drafted token."""
    return -(-(c["q"] if c["op"] == "attend" else c["n"]) // 64)


def _lengths(c):
    """(context lengths, drafted tokens) of each request; for fork the requests' lengths and each new
    request's source. They go by the case alone."""
    r = random.Random(c["shapes"])
    B, ctx = c["B"], c["ctx"]
    if c["op"] == "fork":
        lens = [ctx] * B if c["kind"] == "even" else [r.randint(0, ctx) for _ in range(B)]
        return lens, [i * B // c["n"] for i in range(c["n"])]
    most = c["q"] if c["op"] == "attend" else c["n"]
    if c["kind"] == "even":
        return [ctx] * B, [most] * B
    return [r.randint(0, ctx) for _ in range(B)], [r.randint(1, most) for _ in range(B)]


def _trees(c, n):
    """Each drafted token's parent among its request's (-1: it follows the context)."""
    r = random.Random(c["shapes"] + 1)
    return [[-1 if i == 0 or r.random() < 0.1 else r.randrange(max(0, i - 8), i) for i in range(m)] for m in n]


def _kept(c, n):
    """The drafted tokens of each request that stay, ascending: a node's ancestors and itself, or any."""
    r = random.Random(c["shapes"] + 2)
    out = []
    for p in _trees(c, n):
        if c["kind"] == "any":
            out.append([i for i in range(len(p)) if r.random() < 0.5])
            continue
        at, path = r.randrange(-1, len(p)), []
        while at >= 0:
            path.append(at)
            at = p[at]
        out.append(path[::-1])
    return out


def work(case):
    c = case
    if c["op"] == "rope":
        tokens = c["B"] * c["N"]
        one = 2.0 * tokens * (c["H"] + c["Hkv"]) * c["d"]
        small = 4.0 * c["N"] + 4.0 * min(c["N"], c["top"]) * c["r"]
        # forward: x in, y out; backward: dy and x in, dx out
        return {"bytes": (5 if c["grad"] else 2) * one + small, "flops": (24.0 if c["grad"] else 8.0) * one / 2}
    lens, n = _lengths(c)
    d, bs = c["d"], c["block"]
    if c["op"] == "attend":
        T = sum(n)
        total = sum(lens) + T
        blocks = sum(-(-(x + m) // bs) for x, m in zip(lens, n))
        held = 2.0 * total * c["Hkv"] * d + 2 * 4.0 * blocks * c["Hkv"] + 4.0 * blocks
        depth = 0
        for p in _trees(c, n):
            at = []
            for v in p:
                at.append(1 + (at[v] if v >= 0 else 0))
            depth += sum(at)
        pairs = sum(x * m for x, m in zip(lens, n)) + depth
        return {"bytes": held + T * c["H"] * (4.0 * d + 4) + T * (8.0 + 8.0 * _words(c)) + 12.0 * c["B"],
                "flops": 4.0 * pairs * c["H"] * d}
    if c["op"] == "keep":
        moved = sum(sum(k != i for i, k in enumerate(p)) for p in _kept(c, n))
        return {"bytes": 2.0 * 2 * moved * c["H"] * d + c["B"] * (16.0 + 8.0 * _words(c)), "flops": 0.0}
    part = sum(lens[s] % bs for s in n)
    full = sum(lens[s] // bs for s in n)
    return {"bytes": 2.0 * 2 * part * c["H"] * d + 8.0 * 2 * len(n) * c["H"] + 16.0 * full + 20.0 * len(n),
            "flops": 0.0}


# ------------------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(n):
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    return _ints(cu)


def _need(amax):
    """The smallest power of two s with amax / s <= 448, at least 2^-40."""
    m, e = torch.frexp(amax.float())  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, _LEAST)).clamp(min=_LEAST)
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e)


def _held(gen, blocks, heads, bs, d):
    """Codes and scales of filled blocks: normal values, a size of its own for each head and block."""
    size = torch.exp(0.5 * torch.randn(blocks, heads, 1, 1, device="cuda", generator=gen))
    x = torch.randn(blocks, heads, bs, d, device="cuda", generator=gen) * size
    s = _need(x.abs().amax(dim=(2, 3)))
    return x.div_(s[:, :, None, None]).to(_F8), s


def _tables(c, gen, total, spare):
    """Block ids in random order: each request's blocks in its table row (-1 behind them), then
    `spare` free ones; the number of blocks."""
    bs = c["block"]
    have = [-(-x // bs) for x in total]
    width = max(1, max(have)) + 1
    ids = torch.randperm(sum(have) + spare, device="cuda", generator=gen).to(torch.int32)
    col = torch.arange(width, device="cuda")[None]
    hv = torch.tensor(have, device="cuda")
    first = (torch.cumsum(hv, 0) - hv)[:, None]
    table = torch.where(col < hv[:, None], ids[(first + col).clamp(max=len(ids) - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), ids[sum(have):].contiguous(), len(ids)


def _signed(bits):
    """A set of token numbers as 64-bit words."""
    w = {}
    for i in bits:
        w[i // 64] = w.get(i // 64, 0) | 1 << i % 64
    return w


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "rope":
        return _prepare_rope(c, gen)
    lens, n = _lengths(c)
    bs, d = c["block"], c["d"]
    if c["op"] == "fork":
        table, free, count = _tables(c, gen, lens, c["n"] + 3)
        k, ks = _held(gen, count, c["H"], bs, d)
        v, vs = _held(gen, count, c["H"], bs, d)
        # a draw in some runs out of blocks: the last ones that need one are refused
        if c["shapes"] % 4 == 2:
            free = free[: max(1, (3 * len(free)) // 4)].contiguous()
        return dict(op="fork", block=bs, cache=(k, v, ks, vs), table=table, lens=_ints(lens), src=_ints(n),
                    free=free, pos=_ints([0]), shares=torch.zeros(count, dtype=torch.int32, device="cuda"))
    total = [x + m for x, m in zip(lens, n)]
    heads = c["Hkv"] if c["op"] == "attend" else c["H"]
    table, free, count = _tables(c, gen, total, 3)
    k, ks = _held(gen, count, heads, bs, d)
    v, vs = _held(gen, count, heads, bs, d)
    st = dict(op=c["op"], block=bs, cache=(k, v, ks, vs), table=table, lens=_ints(lens), kv=_ints(total),
              cu=_offsets(n), words=_words(c))
    if c["op"] == "keep":
        words = []
        for p in _kept(c, n):
            w = _signed(p)
            words.append([w.get(i, 0) - (w.get(i, 0) >> 63 << 64) for i in range(st["words"])])
        # the free list: its first entries have been handed out
        used = count - len(free)
        free = torch.cat([torch.full((used,), -1, dtype=torch.int32, device="cuda"), free])
        return dict(st, keep=torch.tensor(words, dtype=torch.int64, device="cuda"), free=free, pos=_ints([used]))
    T = sum(n)
    q = torch.randn(T, c["H"], d, device="cuda", generator=gen).to(_TYPES[c["dtype"]])
    if not c["flat"]:
        q = q.view(c["B"], c["q"], c["H"], d).transpose(1, 2)
    return dict(st, q=q, parents=_ints([v for p in _trees(c, n) for v in p]), flat=c["flat"],
                scale=1.0 / math.sqrt(d), longest=max(total), most=max(n))


def _prepare_rope(c, gen):
    B, N, H, Hkv, d, r = (c[x] for x in ("B", "N", "H", "Hkv", "d", "r"))
    dt = _TYPES[c["dtype"]]

    def make(heads):
        size = torch.exp(0.5 * torch.randn(heads, 1, device="cuda", generator=gen))
        return size, heads

    def rows(sh):
        size, heads = sh
        if c["layout"] == "heads":
            return (torch.randn(B, heads, N, d, device="cuda", generator=gen) * size[:, None]).to(dt)
        return (torch.randn(B, N, heads, d, device="cuda", generator=gen) * size).to(dt).transpose(1, 2)

    if c["layout"] == "fused":  # q, k and v of a token behind one another
        whole = torch.randn(B, N, (H + 2 * Hkv), d, device="cuda", generator=gen).to(dt)
        q, k = whole[:, :, :H].transpose(1, 2), whole[:, :, H:H + Hkv].transpose(1, 2)
    else:
        q, k = rows(make(H)), rows(make(Hkv))
    # the angles in 64 bits, their cosines and sines rounded once
    freq = 10000.0 ** (-torch.arange(r // 2, dtype=torch.float64, device="cuda") * 2 / r)
    angle = torch.arange(c["top"], dtype=torch.float64, device="cuda")[:, None] * freq
    table = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
    first = int(torch.randint(0, max(1, c["top"] - N + 1), (1,), device="cuda", generator=gen))
    at = torch.arange(N, device="cuda") + first
    pos = (at % c["top"]).to(torch.int32)
    wt = torch.float32 if c["weights"] == "fp32" else dt
    w = [None if c["weights"] == "none" else
         (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(wt) for _ in range(2)]
    st = dict(op="rope", q=q, k=k, table=table, pos=pos, wq=w[0], wk=w[1], eps=1e-6, pairs=c["pairs"],
              grad=c["grad"])
    if c["grad"]:
        st["dq"] = rows(make(H)).contiguous() if c["layout"] != "tokens" else rows(make(H))
        st["dk"] = rows(make(Hkv)).contiguous() if c["layout"] != "tokens" else rows(make(Hkv))
    return st


# ------------------------------------------------------------------------------ plain forms

def _split(x, r, pairs):
    """First and second elements of the turned pairs, and the elements behind them."""
    if pairs:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., : r // 2], x[..., r // 2: r], x[..., r:]


def _joined(a, b, rest, pairs):
    ab = torch.stack([a, b], dim=-1).flatten(-2) if pairs else torch.cat([a, b], dim=-1)
    return torch.cat([ab, rest], dim=-1)


def _turned(x, s, back):
    r = s["table"].shape[1]
    rows = s["table"][s["pos"].long()].to(x.dtype)  # [N, r]
    cos, sin = rows[:, : r // 2], rows[:, r // 2:]
    if back:
        sin = -sin
    a, b, rest = _split(x, r, s["pairs"])
    return _joined(a * cos - b * sin, b * cos + a * sin, rest, s["pairs"])


def _rope_plain(s, x, w, g):
    """Result of one of q and k, or with g its gradient and the weights'."""
    f = x.float()
    inv = torch.rsqrt(f.square().mean(-1, keepdim=True) + s["eps"])
    wf = torch.ones(x.shape[-1], device="cuda") if w is None else w.float()
    y = _turned(f * inv * wf, s, False).to(x.dtype)
    if g is None:
        return (y,)
    t = _turned(g.float(), s, True)
    n = f * inv
    dw = (t * n).sum(dim=(0, 1, 2))
    u = t * wf
    dx = inv * (u - n * (u * n).mean(-1, keepdim=True))
    return (y, dx.to(x.dtype)) + (() if w is None else (dw,))


def _tree_plain(s, count, row, there):
    """Which drafted tokens each one sees [B, most, most], from their parents."""
    most = there.shape[1]
    p = torch.where(there, s["parents"].long()[row], -1)
    i = torch.arange(most, device="cuda")
    step = (p[:, :, None] == i) & (p[:, :, None] >= 0) & (i < i[:, None])
    once = step.double() + torch.eye(most, dtype=torch.float64, device="cuda")
    return (torch.linalg.matrix_power(once, 128) > 0) & there[:, :, None]


def _attend_plain(s):
    cu, base, lens = s["cu"].long(), s["lens"].long(), s["kv"].long()
    q = s["q"] if s["flat"] else s["q"].transpose(1, 2).reshape(-1, s["q"].shape[1], s["q"].shape[3])
    T, H, d = q.shape
    B, most = len(lens), s["most"]
    count = cu[1:] - cu[:-1]
    i = torch.arange(most, device="cuda")[None]
    there = i < count[:, None]
    row = (cu[:-1, None] + i).clamp(max=T - 1)
    sees = _tree_plain(s, count, row, there)
    req = torch.repeat_interleave(torch.arange(B, device="cuda"), count, output_size=T)
    at = torch.arange(T, device="cuda") - cu[req]
    bits = torch.nn.functional.pad(sees[req, at], (0, 64 * s["words"] - most)) if 64 * s["words"] >= most \
        else sees[req, at][:, : 64 * s["words"]]
    masks = (bits.reshape(T, -1, 64).long() << torch.arange(64, device="cuda")).sum(-1)
    places = (base[req] + sees[req, at].sum(-1) - 1).to(torch.int32)

    table = s["table"][:, : max(1, -(-s["longest"] // s["block"]))].long().clamp(min=0)
    k, v, ks, vs = s["cache"]
    k, v = _rows_plain(k, ks, table), _rows_plain(v, vs, table)
    heads, keys = k.shape[1], k.shape[2]
    qq = q[row].float().reshape(B, most, heads, H // heads, d).permute(0, 2, 3, 1, 4)
    x = (qq.reshape(B, heads, -1, d) @ k.transpose(2, 3)) * s["scale"]
    x = x.reshape(B, heads, H // heads, most, keys)
    key = torch.arange(keys, device="cuda")
    own_key = key[None] - base[:, None]  # the drafted token that a key belongs to
    drafted = sees.gather(2, own_key.clamp(0, most - 1)[:, None, :].expand(B, most, keys))
    seen = torch.where(own_key[:, None] < 0, there[:, :, None], drafted & (own_key < count[:, None])[:, None])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    ref = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(x - ref)
    total = p.sum(dim=-1, keepdim=True)
    v = torch.where(key[:, None] < lens[:, None, None, None], v, torch.zeros((), device="cuda"))
    o = (p.reshape(B, heads, -1, keys) @ v).reshape(B, heads, H // heads, most, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + ref)[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, most, H, d)[req, at].to(q.dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(B, most, H)[req, at]
    if not s["flat"]:
        o = o.view(B, most, H, d).transpose(1, 2)
        lse = lse.view(B, most, H).transpose(1, 2)
    return masks, places, o, lse


def _rows_plain(codes, scales, table):
    """The cached values [B, heads, keys, d] that a block table lists."""
    B, w = table.shape
    x = codes.view(torch.uint8)[table].view(_F8).float() * scales[table][:, :, :, None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(B, x.shape[2], w * x.shape[3], x.shape[4])


def _moves(s):
    """Kept drafted tokens: their requests, places before and behind; kept ones of each request."""
    keep, lens = s["keep"], s["lens"].long()
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    bits = ((keep[:, :, None] >> torch.arange(64, device="cuda")) & 1).reshape(len(lens), -1)
    bits = bits.bool() & (torch.arange(bits.shape[1], device="cuda") < n[:, None])
    rank = torch.cumsum(bits.long(), 1) - 1
    req, tok = torch.nonzero(bits, as_tuple=True)
    return req, lens[req] + tok, lens[req] + rank[req, tok], bits.sum(1)


def _keep_plain(s):
    table, bs, lens = s["table"].long(), s["block"], s["lens"].long()
    k, v, ks, vs = s["cache"]
    req, at, to, kept = _moves(s)
    for codes, scales in ((k, ks), (v, vs)):
        _move_plain(codes, scales, table[req, at // bs], at % bs, table[req, to // bs], to % bs, lens[req], to, bs)
    after = (lens + kept).to(torch.int32)
    # blocks from the new length's last one on to the old length's, in order, to the free list
    had, has = (s["kv"].long() + bs - 1) // bs, (after.long() + bs - 1) // bs
    col = torch.arange(s["table"].shape[1], device="cuda")
    back = s["table"][(col >= has[:, None]) & (col < had[:, None])]
    where = s["pos"].long() - 1 - torch.arange(len(back), device="cuda")
    s["free"][where] = back
    return k, v, ks, vs, after, s["free"], s["pos"] - len(back)


def _move_plain(codes, scales, b0, r0, b1, r1, base, to, bs):
    raw = codes.view(torch.uint8)
    ids, place = torch.unique(b1, return_inverse=True)
    # rows of each of these blocks that belong to the context
    older = torch.zeros(len(ids), dtype=torch.long, device="cuda")
    older.index_reduce_(0, place, (base - (to - r1)).clamp(min=0), "amax")
    come = scales[b0]
    top = torch.zeros(len(ids), scales.shape[1], device="cuda").index_reduce_(0, place, come, "amax")
    was = scales[ids]
    now = torch.where(older[:, None] > 0, torch.maximum(top, was), top)
    rows = (raw[b0, :, r0].view(_F8).float() * (come / now[place])[:, :, None]).to(_F8).view(torch.uint8)
    held = raw[ids]
    again = (held.view(_F8).float() * (was / now)[:, :, None, None]).to(_F8).view(torch.uint8)
    raw[ids] = torch.where((torch.arange(bs, device="cuda") < older[:, None])[:, None, :, None], again, held)
    raw[b1, :, r1] = rows
    scales[ids] = now


def _fork_plain(s):
    table, bs, src = s["table"], s["block"], s["src"].long()
    lens = s["lens"].long()[src]
    n, width = len(src), table.shape[1]
    part = lens % bs
    upto = torch.cumsum((part > 0).long(), 0)
    ok = (part == 0) | (s["pos"] + upto <= len(s["free"]))
    got = s["free"][(s["pos"].long() + upto - 1).clamp(0, len(s["free"]) - 1)]
    col = torch.arange(width, device="cuda")
    full = (lens // bs)[:, None]
    rows = table[src]
    last = rows.gather(1, full.clamp(max=width - 1))[:, 0]
    out = torch.where((col < full) & ok[:, None], rows, torch.full((), -1, dtype=torch.int32, device="cuda"))
    out = torch.where((col == full) & (ok & (part > 0))[:, None], got[:, None], out)
    shared = rows[(col < full) & ok[:, None]].long()
    s["shares"].index_add_(0, shared, torch.ones(len(shared), dtype=torch.int32, device="cuda"))
    one = (ok & (part > 0))
    copies = torch.where(one[:, None], torch.stack([last, got, part.to(torch.int32)], 1),
                         torch.tensor([-1, -1, 0], dtype=torch.int32, device="cuda"))
    k, v, ks, vs = s["cache"]
    a, b, m = copies[one].long().unbind(1)
    inside = (torch.arange(bs, device="cuda") < m[:, None])[:, None, :, None]
    for codes, scales in ((k, ks), (v, vs)):
        raw = codes.view(torch.uint8)
        raw[b] = torch.where(inside, raw[a], raw[b])
        scales[b] = scales[a]
    used = s["pos"] + one.sum().to(torch.int32)
    return out, torch.where(ok, lens, 0).to(torch.int32), copies, used, s["shares"], k, v, ks, vs


# ------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "rope":
        q = _rope_plain(s, s["q"], s["wq"], s.get("dq"))
        k = _rope_plain(s, s["k"], s["wk"], s.get("dk"))
        return q + k
    return {"attend": _attend_plain, "keep": _keep_plain, "fork": _fork_plain}[s["op"]](s)


def _run_own(s):
    import attention_forward_flashattention_gb300 as fa
    if s["op"] == "rope":
        q, k = fa.qk_norm_rope_forward(s["q"], s["k"], s["table"], s["pos"], s["wq"], s["wk"], eps=s["eps"],
                                       interleaved=s["pairs"])
        if not s["grad"]:
            return q, k
        dq, dk, dwq, dwk = fa.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["table"], s["pos"],
                                                    s["wq"], s["wk"], eps=s["eps"], interleaved=s["pairs"])
        return (q, dq, k, dk) if dwq is None else (q, dq, dwq, k, dk, dwk)
    if s["op"] == "attend":
        masks, places = fa.cache_tree(s["parents"], s["cu"], s["lens"], s["words"])
        o, lse = fa.attention_forward_cache_tree(s["q"], s["cache"], s["table"], s["kv"], masks,
                                                 s["cu"] if s["flat"] else None, scale=s["scale"])
        return masks, places, o, lse
    k, v, ks, vs = s["cache"]
    if s["op"] == "keep":
        after = fa.cache_keep(s["cache"], s["table"], s["kv"], s["cu"], s["keep"])
        pos = fa.cache_release(s["table"], s["kv"], after, s["free"], s["pos"], s["block"])
        return k, v, ks, vs, after, s["free"], pos
    table, lens, copies, pos = fa.cache_fork(s["table"], s["lens"], s["src"], s["free"], s["pos"],
                                             s["shares"], s["block"])
    fa.cache_copy(s["cache"], copies)
    return table, lens, copies, pos, s["shares"], k, v, ks, vs


# ------------------------------------------------------------------------------ 64 bits

def _exact_rope(s, x, w, g):
    f = x.double()
    n = f / torch.sqrt((f * f).sum(-1, keepdim=True) / f.shape[-1] + s["eps"])
    wf = torch.ones(f.shape[-1], dtype=torch.float64, device="cuda") if w is None else w.double()
    r = s["table"].shape[1]
    at = s["table"].double()[s["pos"].long()]
    z = torch.complex(at[:, : r // 2], at[:, r // 2:])

    def turn(t, by):
        a, b, rest = _split(t, r, s["pairs"])
        u = torch.complex(a.contiguous(), b.contiguous()) * by
        return _joined(u.real, u.imag, rest, s["pairs"])
    y = turn(n * wf, z)
    if g is None:
        return (y,)
    t = turn(g.double(), z.conj())
    # y = n w: d n = t w; n = f / rms: its part along n falls away
    dn = t * wf
    rms = f.norm(dim=-1, keepdim=True).square() / f.shape[-1] + s["eps"]
    dx = dn / rms.sqrt() - f * (dn * f).mean(-1, keepdim=True) / rms ** 1.5
    return (y, dx) + (() if w is None else ((t * n).flatten(0, 2).sum(0),))


def _exact_attend(s):
    cu, lens, base, bs = s["cu"].tolist(), s["kv"].tolist(), s["lens"].tolist(), s["block"]
    parents = s["parents"].tolist()
    q = s["q"] if s["flat"] else s["q"].transpose(1, 2).flatten(0, 1)
    T, H, d = q.shape
    k8, v8, ks, vs = s["cache"]
    heads = ks.shape[1]
    g = H // heads
    o = torch.zeros(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    words, places = [], []
    for b, length in enumerate(lens):
        m, sets = cu[b + 1] - cu[b], []
        for i, p in enumerate(parents[cu[b]: cu[b + 1]]):
            sets.append((sets[p] if p >= 0 else frozenset()) | {i})
            places.append(base[b] + len(sets[i]) - 1)
            w = _signed(sets[i])
            words.append([w.get(x, 0) - (w.get(x, 0) >> 63 << 64) for x in range(s["words"])])
        hide = torch.ones(m, length, dtype=torch.bool)
        hide[:, : base[b]] = False
        for i, seen in enumerate(sets):
            hide[i, [base[b] + x for x in seen]] = False
        hide = hide.to("cuda")
        ids = s["table"][b, : -(-length // bs)].long()
        kk, vv = ((c.view(torch.uint8)[ids].view(_F8).double() * f.double()[ids][:, :, None, None])
                  .transpose(0, 1).reshape(heads, -1, d)[:, :length] for c, f in ((k8, ks), (v8, vs)))
        for h in range(heads):
            rows = q[cu[b]: cu[b + 1], h * g: (h + 1) * g].double()
            x = (torch.einsum("mgd,kd->mgk", rows, kk[h]) * s["scale"]).masked_fill(hide[:, None], -math.inf)
            y = torch.logsumexp(x, -1)
            o[cu[b]: cu[b + 1], h * g: (h + 1) * g] = torch.einsum("mgk,kd->mgd", torch.exp(x - y[..., None]), vv[h])
            lse[cu[b]: cu[b + 1], h * g: (h + 1) * g] = y
    if not s["flat"]:
        B = len(lens)
        o, lse = o.view(B, -1, H, d).transpose(1, 2), lse.view(B, -1, H).transpose(1, 2)
    return torch.tensor(words, dtype=torch.int64, device="cuda"), _ints(places), o, lse


def _exact_keep(s):
    """Values before they are rounded to 8 bits again, and everything else as it has to be."""
    table, cu, lens, kv = (s[x].tolist() for x in ("table", "cu", "lens", "kv"))
    bs, keep = s["block"], s["keep"].tolist()
    src, dst, first, after, back = [], [], {}, [], []
    for b, base in enumerate(lens):
        kept = [i for i in range(cu[b + 1] - cu[b]) if keep[b][i // 64] >> i % 64 & 1]
        for j, i in enumerate(kept):
            src.append((table[b][(base + i) // bs], (base + i) % bs))
            dst.append((table[b][(base + j) // bs], (base + j) % bs))
            first[dst[-1][0]] = max(0, base - (base + j) // bs * bs)
        after.append(base + len(kept))
        back += table[b][-(-after[-1] // bs): -(-kv[b] // bs)]
    sb, sr = (torch.tensor([x[i] for x in src], dtype=torch.long, device="cuda") for i in (0, 1))
    tb, tr = (torch.tensor([x[i] for x in dst], dtype=torch.long, device="cuda") for i in (0, 1))
    old = torch.zeros(len(s["cache"][2]), dtype=torch.long, device="cuda")
    hit = torch.zeros(len(old), dtype=torch.bool, device="cuda")
    if first:
        at = torch.tensor(list(first), device="cuda")
        old[at] = torch.tensor(list(first.values()), device="cuda")
        hit[at] = True
    out = []
    for codes, scales in (s["cache"][0::2], s["cache"][1::2]):
        x, f = codes.double(), scales.double()
        blocks, heads = f.shape
        place = (tb[:, None] * heads + torch.arange(heads, device="cuda")).reshape(-1)
        top = torch.zeros(blocks * heads, dtype=torch.float64, device="cuda")
        top.scatter_reduce_(0, place, f[sb].reshape(-1), "amax")
        top = top.view(blocks, heads)
        now = torch.where(hit[:, None], torch.where(old[:, None] > 0, torch.maximum(top, f), top), f)
        rows = x[sb, :, sr] * (f[sb] / now[tb])[:, :, None]
        inside = (torch.arange(bs, device="cuda") < old[:, None])[:, None, :, None] & hit[:, None, None, None]
        x = torch.where(inside, x * (f / now)[:, :, None, None], x)
        x[tb, :, tr] = rows
        out += [x, now]
    free = s["free"].tolist()
    pos = int(s["pos"][0])
    for i, x in enumerate(back):
        free[pos - 1 - i] = x
    return out[0], out[2], out[1], out[3], _ints(after), _ints(free), _ints([pos - len(back)])


def _exact_fork(s):
    table, lens, free, bs = s["table"].tolist(), s["lens"].tolist(), s["free"].tolist(), s["block"]
    shares = s["shares"].tolist()
    rows, got, copies, wanted, used = [], [], [], 0, 0
    for x in s["src"].tolist():
        m = lens[x] % bs
        wanted += m > 0
        ok = m == 0 or wanted <= len(free)
        row = [-1] * len(table[0])
        if ok:
            row[: lens[x] // bs] = table[x][: lens[x] // bs]
            for y in row[: lens[x] // bs]:
                shares[y] += 1
            if m:
                row[lens[x] // bs] = free[used]
                used += 1
        copies.append((table[x][lens[x] // bs], row[lens[x] // bs], m) if ok and m else (-1, -1, 0))
        rows.append(row)
        got.append(lens[x] if ok else 0)
    k, v, ks, vs = (t.clone() for t in s["cache"])
    for a, b, m in copies:
        if m:
            for codes, scales in ((k, ks), (v, vs)):
                codes.view(torch.uint8)[b, :, :m] = codes.view(torch.uint8)[a, :, :m]
                scales[b] = scales[a]
    return (_ints(rows), _ints(got), _ints(copies), _ints([used]), _ints(shares), k.double(), v.double(),
            ks.double(), vs.double())


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return (_exact_rope(s, s["q"], s["wq"], s.get("dq")) + _exact_rope(s, s["k"], s["wk"], s.get("dk")))
    return {"attend": _exact_attend, "keep": _exact_keep, "fork": _exact_fork}[s["op"]](s)
