"""The block cache's upkeep on the GPU against the plain implementations of
pages_util, exactly: kept tokens (codes and scales), the free list, shared blocks,
copies; sizes, layouts and numbers that are out of range; and a serving loop of
drafts, forks and frees whose attention is that of a cache filled afresh."""
import numpy as np
import pytest
import torch

import attention_forward_flashattention_gb300 as fa
import cache_util as U
import draft_util as D
import pages_util as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def make_cache(num, heads, bs, d, layout, rng):
    """A cache of random codes without NaN and of scales that are powers of two."""
    if layout == "head":
        k, v = (torch.zeros(num, heads, bs, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    elif layout == "token":
        k, v = (torch.zeros(num, bs, heads, d, dtype=torch.uint8, device=DEV).transpose(1, 2) for _ in range(2))
    else:
        s = torch.zeros(num, 2, heads, bs, d + 16, dtype=torch.uint8, device=DEV)
        k, v = s[:, 0, :, :, :d], s[:, 1, :, :, :d]
    for t in (k, v):
        c = rng.integers(0, 256, (num, heads, bs, d), dtype=np.uint8)
        t.copy_(torch.from_numpy(np.where((c & 0x7F) == 0x7F, c ^ 1, c).astype(np.uint8)))
    ks, vs = (torch.from_numpy(np.exp2(rng.integers(-9, -4, (num, heads))).astype(np.float32)).to(DEV)
              for _ in range(2))
    return fa.Cache(k, v, ks, vs)


def host(cache):
    """Codes as bytes, and scales."""
    return [(t if t.dtype == torch.float32 else t.view(torch.uint8)).cpu().numpy().copy() for t in cache]


def random_table(rng, lens, bs, num, width):
    table = np.full((len(lens), width), -1, dtype=np.int64)
    ids, at = rng.permutation(num), 0
    for b, x in enumerate(lens):
        m = min(-(-max(x, 0) // bs), width)
        table[b, :m] = ids[at:at + m]
        at += m
    return table, ids[at:]


def same_codes(got, want):
    """Equal but for the sign of NaN."""
    nan = (want & 0x7F) == 0x7F
    return np.array_equal(np.where(nan, 0x7F, got & np.where(nan, 0x7F, 0xFF)), np.where(nan, 0x7F, want))


def check_keep(cache, table, kv, cu, words, bs):
    before = host(cache)
    signed = torch.from_numpy(D.signed(words)).to(DEV)
    out = fa.cache_keep(cache, ints(table), ints(kv), ints(cu), signed)
    after = host(cache)
    for x, s in ((0, 2), (1, 3)):
        codes, scales, lens = P.keep(before[x], before[s], table, kv, cu, words, bs)
        assert same_codes(after[x], codes)
        assert np.array_equal(after[s], scales.astype(np.float32))
    assert out.tolist() == lens
    return out


def random_words(rng, B, words, dense=0.5):
    return [[sum(1 << i for i in range(64) if rng.random() < dense) for _ in range(words)] for _ in range(B)]


# ------------------------------------------------------------ keep

@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,layout,dense", [(1, "head", 0.3), (5, "token", 0.8), (8, "pair", 0.05)])
def test_keep(heads, layout, dense, d, bs):
    rng = np.random.default_rng(bs + d + heads)
    counts = [1, 13, 0, 64, 130, 40, 7, 200]
    base = [0, 15, 9, 100, 3, 64, 1000, 31]
    kv = [x + n for x, n in zip(base, counts)]
    num = sum(-(-x // bs) for x in kv) + 3
    table, _ = random_table(rng, kv, bs, num, max(kv) // bs + 2)
    cache = make_cache(num, heads, bs, d, layout, rng)
    cu = [0, *np.cumsum(counts).tolist()]
    check_keep(cache, table, kv, cu, random_words(rng, len(kv), 4, dense), bs)


@pytest.mark.parametrize("which", ["none", "all", "first", "last", "prefix", "behind"])
def test_keep_extremes(which):
    rng = np.random.default_rng(3)
    counts, base, bs = [40, 64, 1], [10, 0, 15], 16
    kv = [x + n for x, n in zip(base, counts)]
    table, _ = random_table(rng, kv, bs, 20, 8)
    words = {"none": [[0]] * 3, "all": [[2 ** 64 - 1]] * 3, "first": [[1]] * 3,
             "last": [[1 << n - 1] for n in counts], "prefix": [[(1 << n // 2) - 1] for n in counts],
             "behind": [[2 ** 64 - (1 << n) if n < 64 else 0] for n in counts]}[which]
    cache = make_cache(20, 3, bs, 64, "head", rng)
    before = host(cache)
    check_keep(cache, table, kv, [0, 40, 104, 105], words, bs)
    if which in ("none", "all", "first", "prefix", "behind"):   # nothing moves, nothing changes
        assert all(np.array_equal(a, b) for a, b in zip(before, host(cache)))


def test_keep_scales_of_every_kind():
    """Scales that are no power of two, zero, negative, and far apart; NaN codes."""
    rng = np.random.default_rng(4)
    counts, base, bs = [30, 50, 20, 33], [5, 16, 40, 0], 16
    kv = [x + n for x, n in zip(base, counts)]
    table, _ = random_table(rng, kv, bs, 24, 6)
    cache = make_cache(24, 2, bs, 128, "head", rng)
    odd = np.array([0.0, -1.0, 0.3, 1.0, 2.0 ** -30, 5.0, 2.0 ** -40, 0.01], np.float32)
    for s in (cache.k_scales, cache.v_scales):
        s.copy_(torch.from_numpy(rng.choice(odd, (24, 2))))
    cache.k.view(torch.uint8)[:, :, 3, 7] = 0x7F
    cache.v.view(torch.uint8)[:, 1, 9, 100] = 0xFF
    check_keep(cache, table, kv, [0, *np.cumsum(counts).tolist()], random_words(rng, 4, 1), bs)


def test_keep_leaves_what_it_cannot_do():
    """Lengths out of range and blocks that do not exist: the sequence stays as it is."""
    rng = np.random.default_rng(5)
    bs, num = 16, 30
    kv = [20, 5, -3, 100, 40, 60, 1 << 30, 30, 48]
    cu = [0, 10, 20, 22, 30, 28, 48, 50, 60, 70]     # one longer than its sequence, one negative
    table, _ = random_table(rng, [20, 5, 0, 96, 40, 60, 0, 30, 48], bs, num, 6)
    table[5, 3] = -1                                 # within the last 20 of 60
    table[7, 1] = num
    table[8, 0] = -1                                 # before the last 10 of 48: of no account
    cache = make_cache(num, 2, bs, 64, "head", rng)
    out = check_keep(cache, table, kv, cu, random_words(rng, 9, 1), bs)
    assert out.tolist()[1:8] == kv[1:8] and out.tolist()[8] < 48


def test_keep_many_tokens_in_many_words():
    rng = np.random.default_rng(6)
    for bs, base in ((16, 15), (128, 127)):
        kv = [base + 1024, base + 1200]
        num = sum(-(-x // bs) for x in kv)
        table, _ = random_table(rng, kv, bs, num, -(-max(kv) // bs))
        check_keep(make_cache(num, 1, bs, 128, "head", rng), table, kv, [0, 1024, 2224],
                   random_words(rng, 2, 16, 0.7), bs)


# ------------------------------------------------------------ release

def check_release(table, lens, new, free, pos, bs, shares=None):
    f = ints(free)
    sh = None if shares is None else ints(shares)
    nxt = fa.cache_release(ints(table), ints(lens), ints(new), f, ints([pos]), bs, sh)
    want = P.release(np.asarray(table), lens, new, free, pos, bs, shares)
    assert f.tolist() == want[0] and nxt.tolist() == [want[1]]
    if shares is not None:
        assert sh.tolist() == want[2]


@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("B,top,bs", [(1, 0, 16), (1, 100, 16), (1, 20000, 16), (3, 700, 128), (37, 300, 32),
                                      (700, 90, 16), (3000, 40, 16), (40, 9000, 16), (5000, 300, 16)])
def test_release(B, top, bs, counted):
    rng = np.random.default_rng(B + top)
    lens = rng.integers(0, top + 1, B).tolist()
    new = [int(rng.integers(0, x + 1)) if rng.random() < 0.7 else x for x in lens]
    held = sum(-(-x // bs) for x in lens)
    table, _ = random_table(rng, lens, bs, held + 5, top // bs + 2)
    shares = rng.integers(0, 2, held + 5).tolist() if counted else None
    check_release(table, lens, new, [-7] * (held + 5), held, bs, shares)


def test_release_of_shared_blocks():
    """Blocks that several rows of the call hold: once, at the first of them, when the
    last holder is among them; and given up more often than held."""
    rng = np.random.default_rng(8)
    table = rng.integers(0, 40, (60, 9))
    lens, new = [9 * 16] * 60, [0] * 60
    holders = np.bincount(table.ravel(), minlength=40)
    for extra in (-1, 0, 1, 3):
        check_release(table, lens, new, list(range(100, 160)), 50, 16,
                      np.maximum(holders - 1 + extra, 0).tolist())


def test_release_of_shared_blocks_by_many():
    """More entries than one CTA takes at a time, from blocks of few."""
    rng = np.random.default_rng(28)
    table = rng.integers(-2, 3000, (400, 30))
    lens, new = rng.integers(0, 481, 400).tolist(), [0] * 400
    held = np.bincount([x for b in range(400) for x in table[b, :-(-lens[b] // 16)] if x >= 0], minlength=3000)
    shares = np.maximum(held - 1 + rng.integers(-1, 2, 3000), 0)
    check_release(table, lens, new, [-7] * 3100, 3050, 16, shares.tolist())
    check_release(table, lens, new, [-7] * 3100, 17, 16, shares.tolist())


@pytest.mark.parametrize("case", [
    dict(pos=-1), dict(pos=9), dict(pos=0), dict(pos=2),                # no list, no room, too little
    dict(lens=[-4, 50, 5000, 30]), dict(new=[60, -1, 3, 30]),           # numbers out of range
    dict(bad=True), dict(bad=True, shares=[0] * 12)])                   # entries that are no blocks
def test_release_refusals(case):
    table = np.arange(12).reshape(4, 3)
    if case.get("bad"):
        table[1, 1], table[2, 0], table[3, 2] = -1, -2 ** 31, 12 if "shares" in case else 7
    check_release(table, case.get("lens", [48, 20, 17, 30]), case.get("new", [10, 0, 17, 1]), list(range(50, 58)),
                  case.get("pos", 8), 16, case.get("shares"))


# ------------------------------------------------------------ fork and copy

def check_fork(table, lens, src, free, pos, shares, bs):
    sh, tab = ints(shares), ints(table)
    out = fa.cache_fork(tab, ints(lens), ints(src), ints(free), ints([pos]), sh, bs)
    rows, new, copies, nxt, want = P.fork(np.asarray(table), lens, src, free, pos, shares, bs)
    assert np.array_equal(out[0].cpu().numpy(), rows) and out[1].tolist() == new
    assert out[2].tolist() == [list(c) for c in copies] and out[3].tolist() == [nxt]
    assert sh.tolist() == want and np.array_equal(tab.cpu().numpy(), table)
    return out


@pytest.mark.parametrize("B,n,top,bs", [(1, 1, 0, 16), (1, 5, 100, 16), (4, 32, 3000, 128), (20, 700, 50, 32),
                                        (300, 2000, 64, 16), (2, 611, 900, 16), (900, 9001, 40, 16)])
def test_fork(B, n, top, bs):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, top + 1, B).tolist()
    num = sum(-(-x // bs) for x in lens) + n
    table, free = random_table(rng, lens, bs, num, top // bs + 1)
    check_fork(table, lens, rng.integers(0, B, n).tolist(), free.tolist(), 0, rng.integers(0, 3, num).tolist(), bs)


@pytest.mark.parametrize("case", [dict(pos=5), dict(pos=-1), dict(pos=100), dict(free=[]),
                                  dict(src=[-1, 4, 0, 2 ** 31 - 1, -2 ** 31, 1]), dict(lens=[-5, 49, 48, 17]),
                                  dict(entry=-1), dict(entry=30), dict(entry=12)])
def test_fork_refusals(case):
    table = np.arange(12).reshape(4, 3)
    if "entry" in case:
        table[0, 2], table[1, 0] = case["entry"], case["entry"]
    check_fork(table, case.get("lens", [40, 20, 32, 0]), case.get("src", [0, 1, 2, 3, 0, 1, 0]),
               case.get("free", [20, 21, 22, 23, 24, 25, 26]), case.get("pos", 4), [0] * 27, 16)


def test_fork_into_other_rows_of_the_same_table():
    rng = np.random.default_rng(9)
    table = np.full((7, 4), -1, dtype=np.int64)
    table[:2] = rng.permutation(8).reshape(2, 4)
    tab, sh = ints(table), ints([0] * 20)
    lens, copies, nxt = ints([0] * 5), ints(np.zeros((5, 3))), ints([0])
    args = (ints([50, 64] + [0] * 5), ints([0, 1, 0, 0, 1]), ints(range(10, 20)), ints([0]), sh, 16)
    fa.cache_fork(tab, *args, out=(tab[2:], lens, copies, nxt))
    rows, new, cp, n, shares = P.fork(table, [50, 64] + [0] * 5, [0, 1, 0, 0, 1], list(range(10, 20)), 0, [0] * 20, 16)
    assert np.array_equal(tab.cpu().numpy(), np.concatenate([table[:2], rows])) and lens.tolist() == new
    assert copies.tolist() == [list(c) for c in cp] and nxt.tolist() == [n] and sh.tolist() == shares


@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,layout", [(1, "head"), (6, "token"), (3, "pair")])
def test_copy(heads, layout, d, bs):
    rng = np.random.default_rng(bs + d)
    cache = make_cache(40, heads, bs, d, layout, rng)
    want = host(cache)
    ids = rng.permutation(40)
    copies = [(int(ids[i]), int(ids[20 + i]), int(m)) for i, m in
              enumerate([1, bs, bs - 1, bs // 2, 0, -3, 1 << 30, 7])]
    copies += [(-1, 3, 5), (4, -1, 5), (40, 5, 5), (5, 1 << 30, 5), (6, 6, 5), (-1, -1, 0)]
    for a, b, m in copies:
        if 0 <= a < 40 and 0 <= b < 40 and a != b and m > 0:
            for x, s in ((0, 2), (1, 3)):
                want[x][b, :, :min(m, bs)] = want[x][a, :, :min(m, bs)]
                want[s][b] = want[s][a]
    fa.cache_copy(cache, ints(copies))
    assert all(np.array_equal(a, b) for a, b in zip(host(cache), want))


def test_copy_of_nothing_and_of_many():
    rng = np.random.default_rng(11)
    cache = make_cache(4100, 1, 16, 64, "head", rng)
    fa.cache_copy(cache, torch.zeros(0, 3, dtype=torch.int32, device=DEV))
    want = host(cache)
    fa.cache_copy(cache, ints([(i, 2050 + i, 16) for i in range(2050)]))
    want = [np.concatenate([x[:2050], x[:2050]]) for x in want]
    assert all(np.array_equal(a, b) for a, b in zip(host(cache), want))


# ------------------------------------------------------------ streams, graphs, refusals

def test_same_bits_on_streams_and_in_graphs():
    rng = np.random.default_rng(12)
    bs, counts, base = 16, [20, 5, 33], [30, 4, 100]
    kv = [x + n for x, n in zip(base, counts)]
    table, free = random_table(rng, kv, bs, 40, 12)
    cu = ints([0, *np.cumsum(counts).tolist()])
    words = torch.from_numpy(D.signed(random_words(rng, 3, 1))).to(DEV)
    first = make_cache(40, 3, bs, 128, "head", rng)
    tab, kvt, src = ints(table), ints(kv), ints([0, 2, 2])
    lst = ints(np.concatenate([-np.ones(40 - len(free), dtype=np.int64), free]))
    pos = ints([40 - len(free)])

    def step(cache, lst, shares, s=None):
        after = fa.cache_keep(cache, tab, kvt, cu, words, stream=s)
        nxt = fa.cache_release(tab, kvt, after, lst, pos, bs, shares, stream=s)
        new = fa.cache_fork(tab, after, src, lst, nxt, shares, bs, stream=s)
        fa.cache_copy(cache, new[2], stream=s)
        return (after, nxt, *new)

    def state():
        return fa.Cache(*(t.clone() for t in first)), lst.clone(), ints([0] * 40)
    one = state()
    want = step(*one)
    others = [state() for _ in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in others]
    outs = [step(*st, s) for st, s in zip(others, streams)]
    torch.cuda.synchronize()
    for st, out in zip(others, outs):
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip((*st[0], *st[1:]), (*one[0], *one[1:])))
    st = state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*st)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip((*st[0], *st[1:]), (*one[0], *one[1:])))


def test_binding_refuses():
    rng = np.random.default_rng(13)
    cache = make_cache(8, 2, 16, 64, "head", rng)
    t, i2, i3, w = ints(np.zeros((2, 3))), ints([0, 0]), ints([0, 0, 0]), torch.zeros(2, 1, dtype=torch.int64, device=DEV)
    free, pos, sh = ints(range(8)), ints([0]), ints([0] * 8)
    fa.cache_keep(cache, t, i2, i3, w)
    for bad in ((cache, t, i2, i2, w), (cache, t[:1], i2, i3, w), (cache, t.long(), i2, i3, w),
                (cache, t, i2, i3, w.int()), (cache, t, i2, i3, w[:1]), (cache, t, i2, i3, w.cpu()),
                (cache, t.t(), i2, i3, w)):
        with pytest.raises(ValueError):
            fa.cache_keep(*bad)
    with pytest.raises(TypeError):
        fa.cache_keep(cache[:3], t, i2, i3, w)
    for words in (0, 17):
        with pytest.raises(fa.FaError):
            fa.cache_keep(cache, t, i2, i3, torch.zeros(2, words, dtype=torch.int64, device=DEV))
    with pytest.raises(fa.FaError):
        fa.cache_keep(cache, t, i2, i3, w, out=i2)
    for bad in ((t, i2, i3, free, pos, 16), (t, i2, i2.cpu(), free, pos, 16), (t, i2, i2, free[None], pos, 16),
                (t, i2, i2, free, i2, 16), (t, i2, i2, free, pos, 16, sh.long())):
        with pytest.raises(ValueError):
            fa.cache_release(*bad)
    for kw in (dict(block=8), dict(out=pos)):
        with pytest.raises(fa.FaError):
            fa.cache_release(t, i2, i2, free, pos, **{"block": 16, **kw})
    for bad in ((t, i3, i2, free, pos, sh, 16), (t, i2, i2[None], free, pos, sh, 16),
                (t, i2, i2, free.cpu(), pos, sh, 16), (t, i2, i2, free, pos, sh.float(), 16)):
        with pytest.raises(ValueError):
            fa.cache_fork(*bad)
    with pytest.raises(fa.FaError):
        fa.cache_fork(t, i2, i2, free, pos, sh, 17)
    with pytest.raises(fa.FaError):
        fa.cache_fork(t, i2, i2, free, pos, sh, 16, out=(t, i2.clone(), ints(np.zeros((2, 3))), ints([0])))
    for bad in (ints([0, 1, 2]), ints([[0, 1]]), ints([[0, 1, 2]]).long()):
        with pytest.raises(ValueError):
            fa.cache_copy(cache, bad)


# ------------------------------------------------------------ far blocks

def test_blocks_behind_four_gigabytes():
    """Codes whose distance from the cache's start does not fit into 32 bits: attention over
    them, tokens kept in them, blocks copied there, as in a small cache."""
    rng = np.random.default_rng(14)
    bs, heads, d, num = 64, 8, 128, 70000
    counts, base = [20, 70], [100, 64]
    kv = [x + n for x, n in zip(base, counts)]
    table, _ = random_table(rng, kv, bs, 8, 4)
    small = make_cache(8, heads, bs, d, "head", rng)
    far = fa.Cache(*(torch.empty(num, heads, bs, d, dtype=torch.uint8, device=DEV) for _ in range(2)),
                   *(torch.ones(num, heads, device=DEV) for _ in range(2)))
    assert (num - 8) * heads * bs * d > 2 ** 32
    for a, b in zip(far, small):
        a[num - 8:] = b
    words = random_words(rng, 90, 2)
    masks, q = torch.from_numpy(D.signed(words)).to(DEV), torch.randn(90, 16, d, device=DEV).half()
    cu, ftab = ints([0, 20, 90]), np.where(table >= 0, table + num - 8, table)
    for n, rows in ((1, slice(18, 22)), (90, slice(0, 90))):   # the kernels for few rows and for many
        c = cu if n > 1 else ints([0, 2, 4])
        got, want = (fa.attention_forward_cache_tree(q[rows], x, ints(t), ints(kv), masks[rows].contiguous(), c)
                     for x, t in ((far, ftab), (small, table)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    keep = masks[:2].contiguous()
    after = [fa.cache_keep(x, ints(t), ints(kv), cu, keep) for x, t in ((far, ftab), (small, table))]
    assert torch.equal(*after)
    fa.cache_copy(far, ints([(num - 8, num - 9, 33), (num - 7, 5, 64)]))
    for a, b in zip(far, small):
        assert torch.equal(a[num - 8:], b)
    for a, b in zip(far[:2], small[:2]):
        assert torch.equal(a[num - 9, :, :33], b[0, :, :33]) and torch.equal(a[5], b[1])
    for a, b in zip(far[2:], small[2:]):
        assert torch.equal(a[num - 9], b[0]) and torch.equal(a[5], b[1])


# ------------------------------------------------------------ together

@pytest.mark.parametrize("bs,d,H,Hkv,dt", [(16, 64, 4, 2, torch.float16), (32, 128, 8, 1, torch.bfloat16)])
def test_a_serving_loop(bs, d, H, Hkv, dt):
    """Prompts, steps of drafted trees of which a path is kept, a fork of each
    request and its end: the cache holds, within its roundings, what was appended for
    the tokens that each request has, no block is lost, and the attention is that of
    64 bits over what the cache holds."""
    rng = np.random.default_rng(bs)
    num, width, B = 60, 12, 3
    cache = fa.cache_empty(num, Hkv, bs, d, device=DEV)
    table, lens = ints(np.full((B, width), -1)), ints([0] * B)
    free, pos, shares = ints(rng.permutation(num)), ints([0]), ints([0] * num)
    rope = fa.rope_table(1000, d, device=DEV)
    history = [[] for _ in range(B)]   # K and V as they were appended, per token

    def vectors(n):
        return (torch.from_numpy(rng.standard_normal((n, h, d))).to(DEV, dt) for h in (H, Hkv, Hkv))

    for step in range(6):
        counts = [int(rng.integers(1, 30)) if step else int(rng.integers(1, 90)) for _ in range(B)]
        T = sum(counts)
        parents = [i - 1 if step == 0 else (-1 if i == 0 or rng.random() < 0.1 else int(rng.integers(max(0, i - 4), i)))
                   for n in counts for i in range(n)]
        slots, cu, kv, pos = fa.cache_plan(lens, ints(counts), table, free, pos, T, bs)
        words = -(-max(counts) // 64)
        masks, places = fa.cache_tree(ints(parents), cu, lens, words)
        q, k, v = vectors(T)
        q, k = fa.qk_norm_rope_forward(q, k, rope, places)
        fa.cache_append(k, v, slots, cache)
        o, lse = fa.attention_forward_cache_tree(q, cache, table, kv, masks, cu)
        tab, kc, vc, ks, vs = table.cpu().numpy(), *host(cache)
        kvl, cul = kv.tolist(), cu.tolist()
        assert kvl == [x + n for x, n in zip(lens.tolist(), counts)]
        want_masks, want_pos = D.masks_of(parents, cul, lens.tolist(), words)
        assert places.tolist() == want_pos
        eps = torch.finfo(dt).eps
        O, L, to, tl = D.attend(q.double().cpu().numpy(), kc, vc, ks.astype(float),
                                vs.astype(float), tab.astype(np.int64), kvl, cul, want_masks, bs, d ** -0.5, eps,
                                False, 2.0 ** -17)
        assert (np.abs(o.double().cpu().numpy() - O) <= to).all()
        assert (np.abs(lse.double().cpu().numpy() - L) <= tl).all()
        # one path of each request is kept (of the prompt: all of it)
        nodes = [n - 1 if step == 0 else int(rng.integers(0, n)) for n in counts]
        rows = torch.tensor([c + x for c, x in zip(cul, nodes)], device=DEV)
        after = fa.cache_keep(cache, table, kv, cu, masks[rows].contiguous())
        pos = fa.cache_release(table, kv, after, free, pos, bs, shares)
        kf, vf = k.double().cpu().numpy(), v.double().cpu().numpy()
        for b in range(B):
            sets = want_masks[cul[b] + nodes[b]]
            history[b] += [(kf[cul[b] + c], vf[cul[b] + c]) for c in range(counts[b]) if sets[c // 64] >> (c % 64) & 1]
        lens = after
        assert lens.tolist() == [len(h) for h in history]
        if step == 3:   # each request goes on as a copy of another one, the old ones end
            src = [2, 0, 2]
            new, new_lens, copies, pos = fa.cache_fork(table, lens, ints(src), free, pos, shares, bs)
            fa.cache_copy(cache, copies)
            pos = fa.cache_release(table, lens, ints([0] * B), free, pos, bs, shares)
            table, lens, history = new, new_lens, [list(history[s]) for s in src]
        # no block is lost: those held and those free are all blocks, once
        held = {int(x) for b in range(B) for x in table[b, :-(-len(history[b]) // bs)].tolist()}
        left = free.tolist()[pos.tolist()[0]:]
        assert len(left) == len(set(left)) and not held & set(left) and held | set(left) == set(range(num))
        counts_of = np.bincount([x for b in range(B) for x in table[b, :-(-len(history[b]) // bs)].tolist()],
                                minlength=num)
        assert shares.tolist() == np.maximum(counts_of - 1, 0).tolist()
        # what the cache holds of each token: its values, rounded to 8 bits (2^-4 of
        # themselves), once more where its block's scale grew or it moved, or to half of
        # the smallest code, 2^-10, of a scale that leaves the block's largest value below 448
        tab, kc, vc, ks, vs = table.cpu().numpy(), *host(cache)
        for b in range(B):
            for i, (kt, vt) in enumerate(history[b]):
                p, r = tab[b, i // bs], i % bs
                for want, codes, scales in ((kt, kc, ks), (vt, vc, vs)):
                    got = U.CODE_VALUES[codes[p, :, r]] * scales[p][:, None]
                    tol = np.abs(want) * 2.0 ** -4 + scales[p][:, None] * 2.0 ** -10 * 8
                    assert (np.abs(got - want) <= tol).all()
    assert fa.fa_check(int(torch.cuda.current_stream().cuda_stream)) == fa.FA_OK


@pytest.mark.parametrize("back", [0, 5, 16, 21, 32, 40])
@pytest.mark.parametrize("d,dt", [(64, torch.float16), (128, torch.bfloat16)])
def test_a_request_that_goes_back_inside_a_shared_block(d, dt, back):
    """A request of 40 tokens is forked, goes back to an earlier token as a fork of itself, and
    grows by larger values than before: the sibling's tokens keep their codes and scales, no
    block is lost or held twice, and the request has what it kept and what it appended."""
    rng = np.random.default_rng(back + d)
    bs, heads, num, width = 16, 2, 20, 8
    cache = fa.cache_empty(num, heads, bs, d, device=DEV)
    free, pos, shares = ints(rng.permutation(num)), ints([0]), ints([0] * num)
    table, lens = ints(np.full((1, width), -1)), ints([0])

    def grow(table, lens, n, size):
        nonlocal pos
        slots, cu, kv, pos = fa.cache_plan(lens, ints([n]), table, free, pos, n, bs)
        k, v = (torch.from_numpy(size * rng.standard_normal((n, heads, d))).to(DEV, dt) for _ in range(2))
        fa.cache_append(k, v, slots, cache)
        return kv

    def rows(table, n):
        """Values of a request's first n tokens."""
        codes, out = host(cache), []
        for x, s in ((codes[0], codes[2]), (codes[1], codes[3])):
            ids, at = table[0].cpu().numpy()[np.arange(n) // bs], np.arange(n) % bs
            out.append(U.CODE_VALUES[x[ids, :, at]] * s[ids][:, :, None])
        return out

    def account(*held):
        """Blocks held and free are all blocks; counts of holders beside the first one."""
        ids = [int(x) for t, n in held for x in t[0, :-(-n // bs)].tolist()]
        left = free.tolist()[pos.tolist()[0]:]
        assert len(left) == len(set(left)) and not set(ids) & set(left) and set(ids) | set(left) == set(range(num))
        assert shares.tolist() == np.maximum(np.bincount(ids, minlength=num) - 1, 0).tolist()

    lens = grow(table, lens, 40, 1.0)
    sibling, sib_lens, copies, pos = fa.cache_fork(table, lens, ints([0]), free, pos, shares, bs)
    fa.cache_copy(cache, copies)
    account((table, 40), (sibling, 40))
    before = rows(sibling, 40)
    own, own_lens, copies, pos = fa.cache_fork(table, ints([back]), ints([0]), free, pos, shares, bs)
    fa.cache_copy(cache, copies)
    pos = fa.cache_release(table, lens, ints([0]), free, pos, bs, shares)
    account((own, back), (sibling, 40))
    kept = rows(own, back)
    assert all(np.array_equal(a, b[:back]) for a, b in zip(kept, before))
    own_lens = grow(own, own_lens, 30, 500.0)
    assert own_lens.tolist() == [back + 30]
    account((own, back + 30), (sibling, 40))
    after = rows(sibling, 40)
    assert all(np.array_equal(a, b) for a, b in zip(after, before))
    # the kept tokens, rounded once more where their block's scale grew: half of the smallest code of it
    for a, b, s in zip(rows(own, back), kept, host(cache)[2:]):
        if back:
            scale = s[own[0].cpu().numpy()[np.arange(back) // bs]][:, :, None]
            assert (np.abs(a - b) <= scale * 2.0 ** -10 + np.abs(b) * 2.0 ** -4).all()
