"""Trees of drafted tokens on the GPU: masks and positions exactly, the attention
element by element against the 64-bit implementation of draft_util, over head
layouts, types, block sizes, numbers of tokens, masks that leave rows empty, bad
blocks and hidden NaN; chains against the causal attention; streams and graphs."""
import numpy as np
import pytest
import torch

import attention_forward_flashattention_gb300 as fa
import draft_util as D

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def longs(words):
    return torch.from_numpy(D.signed(words)).to(DEV)


def random_parents(rng, counts, reach=6, roots=0.15):
    return [-1 if i == 0 or rng.random() < roots else int(rng.integers(max(0, i - reach), i))
            for n in counts for i in range(n)]


def offsets(counts):
    return [0, *np.cumsum(counts).tolist()]


# ------------------------------------------------------------ masks

@pytest.mark.parametrize("counts,words,spare", [
    ([1], 1, 0), ([5, 0, 64, 1], 1, 3), ([65, 3, 130, 128], 3, 0), ([17] * 300, 1, 0), ([100, 7], 1, 2),
    ([1024], 16, 0), ([1500, 2], 16, 1), ([40], 16, 0)])
def test_masks(counts, words, spare):
    rng = np.random.default_rng(sum(counts))
    T = sum(counts) + spare
    parents = random_parents(rng, counts) + [0] * spare
    cu, lens = offsets(counts), rng.integers(0, 100000, len(counts)).tolist()
    masks = torch.full((T, words), 77, dtype=torch.int64, device=DEV)
    pos = torch.full((T,), 77, dtype=torch.int32, device=DEV)
    fa.cache_tree_into(ints(parents), ints(cu), ints(lens), masks, pos)
    want, wpos = D.masks_of(parents, cu, lens, words)
    want = [[77] * words if m is None else m for m in want]
    assert torch.equal(masks.cpu(), torch.from_numpy(D.signed(want)))
    assert pos.tolist() == [77 if p is None else p for p in wpos]
    again = fa.cache_tree(ints(parents), ints(cu), ints(lens), words)
    used = sum(counts)
    assert torch.equal(again[0][:used], masks[:used]) and torch.equal(again[1][:used], pos[:used])


def test_masks_of_odd_parents_and_lengths():
    parents = [0, 5, -7, 2 ** 31 - 1, 3, -2 ** 31, 4]   # itself, later ones, out of range: no parent
    lens = [-3]
    masks, pos = fa.cache_tree(ints(parents), ints([0, 7]), ints(lens), 1)
    want, wpos = D.masks_of(parents, [0, 7], lens, 1)
    assert masks.tolist() == want and pos.tolist() == wpos
    _, pos = fa.cache_tree(ints([-1, 0]), ints([0, 2]), ints([2 ** 31 - 1]), 1)
    assert pos.tolist() == [2 ** 31 - 1] * 2
    # offsets out of range are clamped, empty ones give nothing
    masks = torch.full((4, 1), 9, dtype=torch.int64, device=DEV)
    fa.cache_tree_into(ints([-1, 0, 1, 2]), ints([-5, 2, 2, 99]), ints([0, 0, 0]), masks,
                       torch.zeros(4, dtype=torch.int32, device=DEV))
    assert masks[:, 0].tolist() == [1, 3, 1, 2]


def test_chain_of_a_thousand():
    masks, pos = fa.cache_tree(ints(range(-1, 1023)), ints([0, 1024]), ints([5]), 16)
    assert pos.tolist() == list(range(5, 1029))
    assert masks[1023].tolist() == [-1] * 16 and masks[64].tolist() == [-1, 1] + [0] * 14


# ------------------------------------------------------------ attention

class Batch:
    """A cache of random codes and scales, block tables in random order, queries and masks."""

    def __init__(self, seed, counts, ctx, H, Hkv, d, bs, dt, kind="tree", words=None, bad=0.0, spare=0,
                 kv=None, uniform=False):
        rng = np.random.default_rng(seed)
        self.counts, self.bs, self.dt, self.scale = counts, bs, dt, 1.3 / d ** 0.5
        self.kv = [c + n for c, n in zip(ctx, counts)] if kv is None else kv
        self.cu = offsets(counts)
        width = max(1, max(-(-x // bs) for x in self.kv)) + 1
        P = sum(-(-max(x, 0) // bs) for x in self.kv) + 2
        ids = rng.permutation(P)
        self.table = np.full((len(counts), width), -1, dtype=np.int64)
        at = 0
        for b, x in enumerate(self.kv):
            m = -(-max(x, 0) // bs)
            self.table[b, :m] = ids[at:at + m]
            at += m
        if bad:
            hit = rng.random(self.table.shape) < bad
            self.table = np.where(hit, rng.choice([-1, -5, P, 1 << 30], self.table.shape), self.table)
        c = rng.integers(0, 256, (2, P, Hkv, bs, d), dtype=np.uint8)
        self.codes = np.where((c & 0x7F) == 0x7F, c ^ 1, c).astype(np.uint8)
        self.scales = np.exp2(rng.integers(-8, -4, (2, P, Hkv))).astype(np.float32)
        self.codes[0] &= 0xBF   # K of moderate size: scores of a few units
        T = self.cu[-1]
        self.words = -(-max(max(counts), 1) // 64) if words is None else words
        if kind == "tree":
            self.masks, _ = D.masks_of(random_parents(rng, counts), self.cu, [0] * len(counts), self.words)
        elif kind == "any":
            self.masks = [[int(rng.integers(0, 2 ** 63)) * 2 + int(rng.integers(0, 2)) for _ in range(self.words)]
                          for _ in range(T)]
        else:
            self.masks = [[0] * self.words for _ in range(T)]
        self.q = torch.from_numpy(rng.standard_normal((T + spare, H, d))).to(DEV, dt)
        self.spare, self.uniform = spare, uniform

    def cache(self):
        k, v = (torch.from_numpy(x).to(DEV) for x in self.codes)
        return fa.Cache(k, v, *(torch.from_numpy(x).to(DEV) for x in self.scales))

    def call(self, cache=None, **kw):
        words = self.masks + [[0] * self.words] * self.spare
        args = (cache or self.cache(), ints(self.table), ints(self.kv), longs(words))
        if self.uniform:
            B = len(self.counts)
            q = self.q.view(B, -1, *self.q.shape[1:]).transpose(1, 2)
            o, lse = fa.attention_forward_cache_tree(q, *args, scale=self.scale, **kw)
            return o.transpose(1, 2).flatten(0, 1), lse.transpose(1, 2).flatten(0, 1)
        return fa.attention_forward_cache_tree(self.q, *args, ints(self.cu), scale=self.scale, **kw)

    def reference(self):
        T = self.cu[-1]
        q = self.q[:T].double().cpu().numpy()
        g = self.q.shape[1] // self.scales.shape[2]
        fp16 = self.dt == torch.float16
        # two parts of a weight: fp16, and every sequence on the kernel for few rows;
        # queries in 8-bit parts: d 128, the kernel for more rows
        two = fp16 and max(self.counts) * g <= 16
        floor = 2.0 ** -17 if q.shape[2] == 128 and max(self.counts) * g > 16 else 0.0
        return D.attend(q, self.codes[0], self.codes[1], self.scales[0].astype(float),
                        self.scales[1].astype(float), self.table, self.kv, self.cu, self.masks, self.bs,
                        self.scale, 2.0 ** -10 if fp16 else 2.0 ** -7, two, floor)

    def check(self):
        o, lse = self.call()
        T = self.cu[-1]
        O, L, to, tl = self.reference()
        got, gl = o[:T].double().cpu().numpy(), lse[:T].double().cpu().numpy()
        none = np.isneginf(L)
        assert np.array_equal(np.isneginf(gl), none) and (got[none] == 0).all()
        over = np.abs(got - O) - to
        assert (over <= 0).all(), f"O {over.max():.3e} over the bound, {(over > 0).sum()} elements"
        over = np.abs(np.where(none, 0, gl) - np.where(none, 0, L)) - tl
        assert (over <= 0).all(), f"LSE {over.max():.3e} over the bound"
        assert fa.fa_check(int(torch.cuda.current_stream().cuda_stream)) == fa.FA_OK
        return o, lse


SHAPES = [
    # counts, contexts, H, Hkv, block
    ([1], [0], 1, 1, 16),
    ([5], [251], 2, 2, 16),
    ([2, 3, 1], [40, 0, 129], 8, 4, 32),                      # the kernel for few rows
    ([4, 4], [700, 333], 4, 1, 128),
    ([7, 12, 3, 1], [100, 260, 0, 1000], 8, 2, 64),           # up to 128 rows, and few
    ([64, 33], [190, 61], 2, 2, 16),
    ([70, 129, 2], [130, 5, 300], 4, 2, 32),                  # more than 64 tokens; pairs of tiles
    ([40, 90], [1, 900], 8, 1, 128),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention(shape, kind, dt, d):
    counts, ctx, H, Hkv, bs = shape
    Batch(sum(counts) + d, counts, ctx, H, Hkv, d, bs, dt, kind).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(1, 1), (2, 4), (9, 1), (13, 8), (40, 4), (130, 2)])
def test_attention_without_offsets(n, group, d):
    Batch(n + d, [n] * 3, [170, 0, 65], 2 * group, 2, d, 32, torch.bfloat16, uniform=True).check()


@pytest.mark.parametrize("group", [1, 3, 6, 16, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_groups(group, d):
    Batch(group, [3, 11], [77, 140], 2 * group, 2, d, 16, torch.float16, "any").check()
    Batch(group, [1, 1, 1], [77, 0, 140], group, 1, d, 16, torch.bfloat16, "any", uniform=True).check()


@pytest.mark.parametrize("counts", [[3, 2], [30, 50], [140, 90]])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing(counts, d):
    """Empty masks: rows with a context see that, rows without one nothing."""
    o, lse = Batch(3, counts, [0, 100], 4, 2, d, 16, torch.float16, "empty").check()
    n = counts[0]
    assert bool((o[:n] == 0).all()) and bool(torch.isneginf(lse[:n]).all())
    assert bool(torch.isfinite(lse[n:]).all())


@pytest.mark.parametrize("kv", [[0, 0, 5], [3, 1, 70], [-4, 1 << 30, 20]])
def test_fewer_keys_than_drafted_tokens(kv):
    """Drafted tokens whose keys would lie before the first one have none; lengths beyond
    the table are taken as its end."""
    b = Batch(7, [6, 40, 21], [0, 0, 0], 4, 2, 128, 16, torch.bfloat16, "any", kv=[min(x, 70) for x in kv])
    b.kv = kv
    b.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("counts", [[4, 1, 3], [20, 60, 9], [150, 100]])
def test_blocks_that_do_not_exist_are_hidden(counts, d):
    Batch(11, counts, [90, 33, 200][:len(counts)], 4, 2, d, 16, torch.float16, "any", bad=0.3).check()


def test_masks_with_too_few_words():
    """Drafted tokens from 64 * words on are seen by nobody."""
    Batch(12, [100, 64, 3], [50, 0, 20], 4, 4, 64, 16, torch.bfloat16, "any", words=1).check()


@pytest.mark.parametrize("group", [1, 4, 12])
def test_few_tokens_of_many_sequences(group):
    """No more tokens than sequences: taken for single tokens, and right if they are not."""
    counts = [0, 0, 5, 0, 1, 0, 0, 0, 2, 0]
    Batch(31 + group, counts, [9, 0, 130, 70, 0, 33, 1, 0, 257, 2], 2 * group, 2, 64, 16, torch.float16).check()


def test_nothing_but_spare_rows():
    b = Batch(33, [0, 0], [5, 40], 4, 2, 128, 16, torch.bfloat16, spare=40, words=1)
    o = torch.full_like(b.q, 7.0)
    lse = torch.full(b.q.shape[:2], 7.0, device=DEV)
    ws = torch.empty(fa.fa_fwd_cache_workspace_size(2, 40, 4, 2, 128), dtype=torch.uint8, device=DEV)
    fa.attention_forward_cache_tree_into(b.q, b.cache(), ints(b.table), ints(b.kv), longs([[0]] * 40), o, lse, ws,
                                         ints([0, 0, 0]))
    assert bool((o == 7).all()) and bool((lse == 7).all())


def test_sixteen_words():
    Batch(13, [1024], [100], 1, 1, 64, 128, torch.bfloat16, "any", words=16).check()


@pytest.mark.parametrize("counts,group", [([5, 3], 2), ([30, 40], 2), ([100, 140], 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_nan(counts, group, d):
    """NaN in K and V of drafted keys reaches the rows that see them and no other."""
    b = Batch(14, counts, [70, 140], 2 * group, 2, d, 16, torch.bfloat16, "tree")
    clean = b.check()
    cache = b.cache()
    seq, c, col = 1, counts[1] // 2, 17
    key = b.kv[seq] - counts[seq] + c
    page, row = b.table[seq, key // 16], key % 16
    cache.v.view(torch.uint8)[page, 0, row, col] = 0x7F
    cache.k.view(torch.uint8)[page, 1, row, col] = 0xFF
    o, lse = b.call(cache)
    sees = np.zeros(b.cu[-1], dtype=bool)
    for i in range(counts[seq]):
        sees[b.cu[seq] + i] = b.masks[b.cu[seq] + i][c // 64] >> (c % 64) & 1
    sees = torch.from_numpy(sees).to(DEV)
    head0, head1 = slice(0, group), slice(group, 2 * group)
    # head 0: V's column
    nan = torch.isnan(o[:, head0])
    assert bool(nan[sees][..., col].all()) and int(nan.sum()) == int(sees.sum()) * group
    assert torch.equal(torch.where(nan, clean[0][:, head0], o[:, head0]), clean[0][:, head0])
    assert torch.equal(lse[:, head0], clean[1][:, head0])
    # head 1: K, the whole row
    assert bool(torch.isnan(o[:, head1][sees]).all()) and bool(torch.isnan(lse[:, head1][sees]).all())
    assert torch.equal(o[:, head1][~sees], clean[0][:, head1][~sees])
    assert torch.equal(lse[:, head1][~sees], clean[1][:, head1][~sees])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("counts", [[4, 6], [40, 30], [140, 130]])
def test_query_rows_that_are_not_finite(counts, bad):
    """Such a row is NaN where it sees a key, nothing where it sees none, and reaches no other."""
    b = Batch(15, counts, [0, 60], 2, 2, 128, 16, torch.float16, "empty")
    b.masks[1] = [1] + b.masks[1][1:]
    clean = b.check()
    for t in (0, 1, b.cu[1] + 1):
        b.q[t, 0, 5] = bad
    o, lse = b.call()
    assert bool((o[0, 0] == 0).all()) and bool(torch.isneginf(lse[0, 0]))
    assert bool(torch.isnan(o[1, 0]).all()) and bool(torch.isnan(o[b.cu[1] + 1, 0]).all())
    keep = torch.ones(o.shape[:2], dtype=torch.bool, device=DEV)
    for t in (0, 1, b.cu[1] + 1):
        keep[t, 0] = False
    assert torch.equal(o[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


def test_rows_behind_the_last_sequence_are_left():
    b = Batch(16, [3, 20], [50, 90], 4, 2, 64, 16, torch.float16, spare=5)
    o = torch.full_like(b.q, 7.0)
    lse = torch.full(b.q.shape[:2], 7.0, device=DEV)
    ws = torch.empty(fa.fa_fwd_cache_workspace_size(2, 28, 4, 2, 64), dtype=torch.uint8, device=DEV)
    fa.attention_forward_cache_tree_into(b.q, b.cache(), ints(b.table), ints(b.kv), longs(b.masks + [[0]] * 5),
                                         o, lse, ws, ints(b.cu), scale=b.scale)
    want = b.check()
    assert torch.equal(o[:23], want[0][:23]) and torch.equal(lse[:23], want[1][:23])
    assert bool((o[23:] == 7).all()) and bool((lse[23:] == 7).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts", [[1, 4, 2], [3, 30, 17], [200, 60], [9] * 40])
def test_chains_are_the_causal_attention(counts, dt, d):
    """Bit for bit: the same kernels with the same keys seen."""
    ctx = [(97 * i) % 400 for i in range(len(counts))]
    b = Batch(17, counts, ctx, 4, 2, d, 32, dt)
    parents = [i - 1 for n in counts for i in range(n)]
    masks, pos = fa.cache_tree(ints(parents), ints(b.cu), ints(ctx), b.words)
    cache, table, kv, cu = b.cache(), ints(b.table), ints(b.kv), ints(b.cu)
    got = fa.attention_forward_cache_tree(b.q, cache, table, kv, masks, cu, scale=b.scale)
    want = fa.attention_forward_cache(b.q, cache, table, kv, cu, causal=True, scale=b.scale)
    assert pos.tolist() == [c + i for c, n in zip(ctx, counts) for i in range(n)]
    eps = torch.finfo(dt).eps
    assert torch.allclose(got[0].float(), want[0].float(), rtol=2 * eps, atol=2 * eps * 8)
    assert torch.allclose(got[1], want[1], rtol=1e-5, atol=1e-5)


def test_long_context_in_many_shares():
    """Sequences that many CTAs share: partial results of tiles with and without drafted keys."""
    for n, dt in ((3, torch.bfloat16), (24, torch.float16)):
        Batch(18 + n, [n, 2], [9000, 1], 4, 2, 128, 128, dt).check()


def test_many_sequences_of_odd_sizes():
    rng = np.random.default_rng(21)
    counts = rng.integers(0, 30, 50).tolist()
    Batch(19, counts, rng.integers(0, 300, 50).tolist(), 4, 2, 64, 16, torch.bfloat16).check()


def test_same_call_same_bits_on_streams_and_in_graphs():
    b = Batch(20, [5, 70, 2], [300, 100, 1000], 8, 2, 128, 32, torch.bfloat16)
    cache, table, kv, cu = b.cache(), ints(b.table), ints(b.kv), ints(b.cu)
    parents = ints(random_parents(np.random.default_rng(5), b.counts))
    lens = kv - (cu[1:] - cu[:-1])

    def step(s=None):
        masks, pos = fa.cache_tree(parents, cu, lens, b.words, stream=s)
        return (masks, pos, *fa.attention_forward_cache_tree(b.q, cache, table, kv, masks, cu, stream=s))
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [step(s) for s in streams]
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for shift in (0, 1):
        parents.copy_(torch.clamp(parents - shift, min=-1))
        want = step()
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_binding_refuses():
    b = Batch(22, [3, 4], [20, 30], 4, 2, 64, 16, torch.float16)
    cache, table, kv, cu, masks = b.cache(), ints(b.table), ints(b.kv), ints(b.cu), longs(b.masks)
    call = fa.attention_forward_cache_tree
    call(b.q, cache, table, kv, masks, cu)
    for m in (masks.int(), masks[:-1], masks[:, 0], masks.cpu(), masks.t(), masks.view(1, 7, 1)):
        with pytest.raises(ValueError):
            call(b.q, cache, table, kv, m, cu)
    with pytest.raises(fa.FaError):
        call(b.q, cache, table, kv, masks.expand(7, 1).repeat(1, 17), cu)
    with pytest.raises(fa.FaError):
        call(b.q, cache, table, kv, masks[:, :0], cu)
    with pytest.raises(TypeError):
        call(b.q, cache, table, kv, None, cu)
    p = ints([-1] * 7)
    for bad in ((p.long(), cu, kv), (p, cu[:-1], kv), (p, cu, kv.cpu()), (p[None], cu, kv)):
        with pytest.raises(ValueError):
            fa.cache_tree(*bad)
    for words in (0, 17, -1):
        with pytest.raises(fa.FaError):
            fa.cache_tree(p, cu, kv, words)
    with pytest.raises(ValueError):
        fa.cache_tree_into(p, cu, kv, masks.int(), p.clone())


def test_no_tokens():
    b = Batch(23, [2], [9], 2, 2, 64, 16, torch.float16)
    none = torch.zeros(0, 2, 64, dtype=torch.float16, device=DEV)
    masks, pos = fa.cache_tree(ints([]), ints([0, 0]), ints([9]))
    assert masks.shape == (0, 1) and pos.shape == (0,)
    o, lse = fa.attention_forward_cache_tree(none, b.cache(), ints(b.table), ints(b.kv), masks, ints([0, 0]))
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
