"""Many items to a CTA of the kernel for many rows: sequences without keys between
others, and trees of many sizes whose shares hold several items and cut some of them,
element by element against the 64-bit implementation; NaN in drafted keys; chains
by their masks and by the causal rule."""
import numpy as np
import pytest
import torch

import attention_forward_flashattention_gb300 as fa
import draft_util as D
from test_gpu_draft import Batch, ints, longs, offsets

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("d,group", [(64, 1), (64, 7), (128, 1), (128, 7)])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tree", [False, True])
def test_nan_on_both_sides_of_sequences_without_keys(tree, dt, d, group):
    """Every other sequence has no keys, so that the last of seven heads of one with keys and
    the first head of the next one are eight items apart, with no tile between them. All
    have NaN in the same column of V: the rows that see it are NaN there."""
    B, n, bs, heads = 8 * sms(), 20, 32, 7
    rng = np.random.default_rng(d + group)
    full = np.arange(B) % 2 == 0
    table = np.where(full, np.cumsum(full) - 1, -1)[:, None]
    P = int(full.sum())
    codes = rng.integers(0, 0x70, (2, P, heads, bs, d), dtype=np.uint8)
    k, v = (torch.from_numpy(c).to(DEV) for c in codes)
    cache = fa.Cache(k, v, *(torch.full((P, heads), 2.0 ** -6, device=DEV) for _ in range(2)))
    q = torch.from_numpy(rng.standard_normal((B, heads * group, n, d))).to(DEV, dt)
    lens = ints(np.where(full, n, 0))

    def call():
        if not tree:
            return fa.attention_forward_cache(q, cache, ints(table), lens)
        chain = torch.from_numpy((np.int64(2) << np.arange(n)) - 1).to(DEV)
        return fa.attention_forward_cache_tree(q, cache, ints(table), lens,
                                               chain[None, :, None].expand(B, n, 1).contiguous())
    clean = call()
    assert bool(torch.isfinite(clean[0]).all())
    v[:, :, 1, 17] = 0x7F   # token 1: every row but the first sees it
    o, lse = call()
    want = clean[0].clone()
    want[::2, :, 1:, 17] = float("nan")
    bad = torch.isnan(o) != torch.isnan(want)
    assert not bool(bad.any()), f"{int(bad.sum())} of {int(torch.isnan(want).sum())} elements"
    assert torch.equal(o.nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(lse, clean[1])


def odd_batch(seed, d, dt, kind="tree"):
    """170 trees over contexts of 0 to 600 keys, some of no keys at all, of more than 128 rows, of a
    context of many tiles: some 50 counted tiles and several items to a CTA, cut items among them."""
    rng = np.random.default_rng(seed)
    counts = rng.integers(1, 65, 170).tolist()
    ctx = rng.integers(0, 601, 170).tolist()
    for b in (7, 90, 133):
        counts[b] = 140
    ctx[40] = 6000
    kv = [c + n for c, n in zip(ctx, counts)]
    for b in [*range(20, 30), 60, 61, 100, 169]:
        kv[b] = 0
    return Batch(seed, counts, ctx, 8, 4, d, 16, dt, kind, kv=kv)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_many_items_of_a_cta(dt, d):
    b = odd_batch(51 + d, d, dt)
    o, lse = b.check()
    again = b.call()
    T = b.cu[-1]
    assert torch.equal(again[0][:T], o[:T]) and torch.equal(again[1][:T], lse[:T])

    # some of the sequences by themselves: within the bounds of both calls
    O, L, to, tl = b.reference()
    cache = b.cache()
    for s in (7, 40, 100, 168):
        rows = slice(b.cu[s], b.cu[s + 1])
        one = fa.attention_forward_cache_tree(b.q[rows].contiguous(), cache, ints(b.table[s:s + 1]),
                                              ints(b.kv[s:s + 1]), longs(b.masks[rows]),
                                              ints([0, b.counts[s]]), scale=b.scale)
        assert (np.abs(one[0].double().cpu().numpy() - O[rows]) <= to[rows]).all()
        assert torch.equal(torch.isneginf(one[1]), torch.isneginf(lse[rows]))


@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_many_items_of_a_cta(d):
    """NaN in V of a drafted key of every sequence that has keys, head by head in other
    columns: the rows that see it are NaN there, all others as without it."""
    b = odd_batch(77, d, torch.bfloat16)
    cache = b.cache()
    clean = b.call(cache)
    want = torch.zeros_like(clean[0], dtype=torch.bool)
    view = cache.v.view(torch.uint8)
    for s, n in enumerate(b.counts):
        if b.kv[s] == 0:
            continue
        c, h, col = n // 2, s % 4, (3 * s) % d
        key = b.kv[s] - n + c
        view[int(b.table[s, key // 16]), h, key % 16, col] = 0xFF
        rows = [b.cu[s] + i for i in range(n) if b.masks[b.cu[s] + i][c // 64] >> (c % 64) & 1]
        want[rows, 2 * h:2 * h + 2, col] = True
    o, lse = b.call(cache)
    assert torch.equal(torch.isnan(o), want)
    assert torch.equal(torch.where(want, 0, o), torch.where(want, 0, clean[0])) and torch.equal(lse, clean[1])

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts", [[1, 4, 2], [3, 30, 17], [200, 60], [9] * 40])
def test_chains_and_the_causal_attention_within_bounds(counts, dt, d):
    """The masks of chains and the causal rule, each element by element: the two calls may
    take other kernels and cuts, so they agree within their bounds."""
    ctx = [(97 * i) % 400 for i in range(len(counts))]
    b = Batch(17, counts, ctx, 4, 2, d, 32, dt)
    b.masks, _ = D.masks_of([i - 1 for n in counts for i in range(n)], offsets(counts), ctx, b.words)
    b.check()
    o, lse = fa.attention_forward_cache(b.q, b.cache(), ints(b.table), ints(b.kv), ints(b.cu), causal=True,
                                        scale=b.scale)
    O, L, to, tl = b.reference()
    assert (np.abs(o.double().cpu().numpy() - O) <= to).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= tl).all()


@pytest.mark.parametrize("counts", [[1], [64], [65], [3, 70], [40, 40], [200, 1], [1024], [1500]])
def test_masks_hold_all_tokens_without_being_told(counts):
    """cache_tree without a number of words hides no token of up to 1024: each sees itself."""
    T = sum(counts)
    parents = [-1 if i == 0 else i // 2 for n in counts for i in range(n)]
    cu, lens = offsets(counts), [7] * len(counts)
    masks, pos = fa.cache_tree(ints(parents), ints(cu), ints(lens))
    words = min(-(-T // 64), 16)
    want, wpos = D.masks_of(parents, cu, lens, words)
    assert masks.shape == (T, words)
    assert torch.equal(masks.cpu(), torch.from_numpy(D.signed(want))) and pos.tolist() == wpos
