"""The block cache's attention judged result by result: every element of O
against a bound made of that element's own terms (cache_util.attend_columns), so
that weights far below a row's largest one, lost partial results and wrong
columns show beside large neighbours."""
import numpy as np
import pytest

import attention_forward_flashattention_gb300 as fa
import cache_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# rows to the one K / V head, head dimension: the step kernel's two instances, and
# the chunk kernel on items of 128 rows (d = 128: queries in 8-bit parts; d = 64) and 256
KERNELS = [(1, 64), (1, 128), (12, 64), (12, 128), (24, 64), (24, 128), (150, 64), (150, 128)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def ints(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def tdt(name):
    import torch
    return torch.float16 if name == "fp16" else torch.bfloat16


def to_cache(k, v, ks, vs):
    import torch
    return fa.Cache(*(torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in (k, v)),
                    *(torch.from_numpy(np.asarray(x, dtype=np.float32)).to(DEV) for x in (ks, vs)))


def two_parts(rows, dtype):
    """Whether a call of so many rows to a K / V head keeps its weights in two fp16 parts."""
    return dtype == "fp16" and rows <= 16


def compare(q, cache, table, lens, cu, causal=True, scale=None, dtype="bf16", two=False, q_floor=0.0):
    """Runs the call and judges every element of O and LSE. q: CUDA tensor [T, H, d]."""
    import torch
    d, bs = q.shape[2], cache.k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o, lse = fa.attention_forward_cache(q, cache, ints(table), ints(lens), ints(cu), causal, scale)
    assert fa.fa_check(0) == fa.FA_OK
    host = [c.view(torch.uint8).cpu().numpy() for c in cache[:2]]
    O, L, tol_o, tol_l = U.attend_columns(
        q.double().cpu().numpy(), *host, *(s.double().cpu().numpy() for s in cache[2:]),
        np.asarray(table), lens, cu, bs, scale, causal, torch.finfo(tdt(dtype)).eps, two, q_floor)
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(gl), empty) and np.all(got[empty] == 0)
    err = np.abs(got - O)
    assert np.all(err <= tol_o), f"O: {np.max(err / tol_o):.2f} of the bound"
    le = np.abs(gl - L)[~empty] / tol_l[~empty]
    assert np.all(le <= 1), f"LSE: {np.max(le):.2f} of the bound"
    return o, lse


def codes(values, shape):
    return U.encode(np.broadcast_to(np.asarray(values, dtype=np.float64), shape))


# ------------------------------------------------------------ weights far below the largest one

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,d", KERNELS)
@pytest.mark.parametrize("apart", [8, 18, 24, 26])
def test_small_scale_block_beside_a_large_one(n, d, dtype, apart):
    """Two blocks of 16 keys that follow each other eight times, with equal scores, V
    scales 2^apart and 1. Columns below 32 are zero in the block of the large scale:
    there O is half of the other block's 256, although its weights are 2^-apart of
    the large ones."""
    import torch
    bs = 16
    k = np.zeros((2, 1, bs, d), np.uint8)
    big = np.where(np.arange(d) < 32, 0.0, 1.0)
    v = np.stack([codes(big, (1, bs, d)), codes(256.0, (1, bs, d))])
    cache = to_cache(k, v, np.ones((2, 1)), [[2.0 ** apart / (4096.0 if dtype == "fp16" else 1.0)],
                                             [1.0 / (4096.0 if dtype == "fp16" else 1.0)]])
    q = torch.randn(n, 1, d, device=DEV).to(tdt(dtype))
    o, _ = compare(q, cache, [[0, 1] * 8], [256], [0, n], False, dtype=dtype, two=two_parts(n, dtype))
    assert torch.all(o[:, :, :32] != 0)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,d", KERNELS)
@pytest.mark.parametrize("nats", [10.0, 18.0])
def test_many_small_weights_beside_one_large(n, d, dtype, nats):
    """20000 keys of V = 1 and one, `nats` ahead of them, of V = 0: O is the share
    of the many, 20000 e^-nats / (1 + 20000 e^-nats)."""
    import torch
    bs, keys = 64, 20001
    P = -(-keys // bs)
    k = np.zeros((P, 1, bs, d), np.uint8)
    v = codes(1.0, (P, 1, bs, d)).copy()
    k[P // 2, 0, 7, 0] = U.encode(np.array([1.0]))[0]
    v[P // 2, 0, 7] = 0
    cache = to_cache(k, v, np.ones((P, 1)), np.ones((P, 1)))
    q = torch.zeros(n, 1, d, device=DEV, dtype=tdt(dtype))
    q[:, :, 0] = nats
    compare(q, cache, np.arange(P)[None], [keys], [0, n], False, 1.0, dtype, two_parts(n, dtype))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,d", KERNELS)
def test_random_values_column_by_column(n, d, dtype):
    """Normal values, sharp scores, scales 2^-12 to 1 apart, ragged keys."""
    import torch
    rng = np.random.default_rng(n + d)
    bs, keys = 32, n + 603
    P = -(-keys // bs)
    k, v = (U.encode(rng.standard_normal((P, 1, bs, d)) * 64) for _ in range(2))
    cache = to_cache(k, v, np.exp2(rng.integers(-7, -4, (P, 1))), np.exp2(rng.integers(-12, 1, (P, 1))))
    q = torch.from_numpy(rng.standard_normal((n, 1, d)) * 2).to(DEV).to(tdt(dtype))
    floor = 2.0 ** -17 if d == 128 and 16 < n <= 128 else 0.0
    compare(q, cache, rng.permutation(P)[None], [keys], [0, n], True, None, dtype,
            two_parts(n, dtype), floor)


# ------------------------------------------------------------ queries without a value

def small_cache(rng, P, heads, bs, d):
    k, v = (U.encode(rng.standard_normal((P, heads, bs, d)) * 64) for _ in range(2))
    return to_cache(k, v, *(np.exp2(rng.integers(-8, -5, (P, heads))) for _ in range(2)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,d", KERNELS)
def test_queries_without_a_value_that_see_no_key(n, d, dtype):
    """More query rows than keys: rows with an infinity or NaN that see no key give
    O = 0 and LSE = -inf like any other, those that see one give NaN; with all blocks
    hidden none sees a key. Rows beside them keep their bits."""
    import torch
    rng = np.random.default_rng(n + d)
    keys = max(n - 6, 0)
    cache = small_cache(rng, 12, 1, 16, d)
    table = ints(rng.permutation(12)[None])
    q = torch.from_numpy(rng.standard_normal((n, 1, d))).to(DEV).to(tdt(dtype))
    clean, cl = fa.attention_forward_cache(q, cache, table, ints([keys]), ints([0, n]))
    bad = [r for r in (0, 1, 2, 7, 8, n - 1) if r < n]
    for r, x in zip(bad, [float("nan"), float("inf"), -float("inf")] * 2):
        q[r, 0, (5 * r) % d] = x
    o, lse = fa.attention_forward_cache(q, cache, table, ints([keys]), ints([0, n]))
    sees = torch.arange(n, device=DEV) >= n - keys
    nan = torch.zeros(n, dtype=torch.bool, device=DEV)
    nan[bad] = True
    assert (o[~sees] == 0).all() and torch.isneginf(lse[~sees]).all()
    assert torch.isnan(o[sees & nan]).all() and not torch.isfinite(lse[sees & nan]).any()
    assert torch.equal(o[~nan], clean[~nan]) and torch.equal(lse[~nan], cl[~nan])
    for hidden in (torch.full_like(table, -1), torch.full_like(table, 12)):
        o, lse = fa.attention_forward_cache(q, cache, hidden, ints([192]), ints([0, n]))
        assert (o == 0).all() and torch.isneginf(lse).all()
    assert fa.fa_check(0) == fa.FA_OK


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,d", KERNELS)
@pytest.mark.parametrize("hidden", [40, 3000])
def test_queries_without_a_value_over_hidden_blocks(n, d, hidden, dtype):
    """The first blocks of a sequence are hidden up to a key that only the later rows
    see past: rows of NaN before it see nothing, those behind it give NaN, also where
    the hidden keys and the others are other CTAs' shares."""
    import torch
    rng = np.random.default_rng(n + d)
    first, bs = 16 * (hidden // 16), 16
    keys = first + max(n // 2, 1)                     # row i sees keys - n + i + 1 of them
    P = -(-keys // bs)
    cache = small_cache(rng, P, 1, bs, d)
    table = rng.permutation(P)[None]
    table[0, :first // bs] = np.where(np.arange(first // bs) % 2, -1, P)
    q = torch.from_numpy(rng.standard_normal((n, 1, d))).to(DEV).to(tdt(dtype))
    q[::2, 0, 1] = float("nan")
    o, lse = fa.attention_forward_cache(q, cache, ints(table), ints([keys]), ints([0, n]))
    nan = torch.arange(n, device=DEV) % 2 == 0
    sees = torch.arange(n, device=DEV) + keys - n + 1 > first
    assert (o[~sees] == 0).all() and torch.isneginf(lse[~sees]).all()
    assert torch.isnan(o[sees & nan]).all() and not torch.isfinite(lse[sees & nan]).any()
    assert torch.isfinite(o[sees & ~nan]).all() and torch.isfinite(lse[sees & ~nan]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,d", KERNELS)
def test_infinite_queries_whose_scores_are_all_minus_infinity(n, d, dtype):
    """An infinity against keys of one sign: every score is -inf, whose softmax has no
    value (and it is not a row without keys)."""
    import torch
    rng = np.random.default_rng(n)
    cache = small_cache(rng, 30, 1, 32, d)
    cache.k.fill_(int(U.encode(np.array([-2.0]))[0]))
    q = torch.from_numpy(rng.standard_normal((n, 1, d))).to(DEV).to(tdt(dtype))
    q[n // 2, 0, 3] = float("inf")
    o, lse = fa.attention_forward_cache(q, cache, ints(np.arange(30)[None]), ints([901]), ints([0, n]))
    bad = torch.arange(n, device=DEV) == n // 2
    assert torch.isnan(o[bad]).all() and not torch.isfinite(lse[bad]).any()
    assert torch.isfinite(o[~bad]).all() and torch.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("n,d", KERNELS)
def test_queries_whose_factor_underflows(n, d):
    """bf16 queries of 2^-120 over K scales of 2^-40: scores of nothing, so O is the
    mean of the values that a row sees, and hidden keys stay hidden."""
    import torch
    rng = np.random.default_rng(n + d)
    cache = small_cache(rng, 20, 1, 16, d)
    cache.k_scales.fill_(2.0 ** -40)
    q = torch.from_numpy(rng.standard_normal((n, 1, d)) * 2.0 ** -120).to(DEV).to(torch.bfloat16)
    keys = n + 97
    compare(q, cache, rng.permutation(20)[None], [keys], [0, n], True, None, "bf16")


# ------------------------------------------------------------ the scales' range

@pytest.mark.parametrize("n,d", KERNELS)
@pytest.mark.parametrize("low,high", [(-60, -55), (-60, 30), (-30, 60), (20, 110), (105, 110)])
def test_v_scales_at_the_ends_of_their_range(n, d, low, high):
    """V scales that are no powers of two, at either end of the documented range and up
    to 2^90 apart; results in bf16, which holds them all."""
    import torch
    rng = np.random.default_rng(n + d)
    bs, P = 16, 40
    k = U.encode(rng.standard_normal((P, 1, bs, d)) * 64)
    v = U.encode(rng.standard_normal((P, 1, bs, d)) * 64)
    vs = np.exp2(rng.uniform(low, high, (P, 1)))
    vs[3], vs[7] = np.exp2(low) * 1.01, np.exp2(high) * 0.99
    cache = to_cache(k, v, np.exp2(rng.uniform(-8, -5, (P, 1))), vs)
    q = torch.from_numpy(rng.standard_normal((n, 1, d))).to(DEV).to(torch.bfloat16)
    floor = 2.0 ** -17 if d == 128 and 16 < n <= 128 else 0.0
    compare(q, cache, rng.permutation(P)[None], [bs * P - 5], [0, n], True, None, "bf16", False, floor)


@pytest.mark.parametrize("n,d", KERNELS)
@pytest.mark.parametrize("e", [-60, -31, 50])
def test_k_scales_at_the_ends_of_their_range(n, d, e):
    """K scales near 2^e, and queries that bring the scores back to ordinary sizes."""
    import torch
    rng = np.random.default_rng(n + d)
    bs, P = 32, 20
    k, v = (U.encode(rng.standard_normal((P, 1, bs, d)) * 64) for _ in range(2))
    cache = to_cache(k, v, np.exp2(e + rng.uniform(0, 2, (P, 1))), np.ones((P, 1)))
    q = torch.from_numpy(rng.standard_normal((n, 1, d)) * 2.0 ** (-e - 7)).to(DEV).to(torch.bfloat16)
    floor = 2.0 ** -17 if d == 128 and 16 < n <= 128 else 0.0
    compare(q, cache, rng.permutation(P)[None], [bs * P - 5], [0, n], True, None, "bf16", False, floor)


# ------------------------------------------------------------ split and joined

def keys_of(rng, P, heads, bs, d):
    """Codes with values that differ from column to column and along the keys, so that a
    lost or misplaced share changes every column."""
    k = U.encode(rng.standard_normal((P, heads, bs, d)) * 32)
    lift = np.arange(P)[:, None, None, None] / P + np.arange(d) / d
    v = U.encode((rng.standard_normal((P, heads, bs, d)) * 0.25 + lift) * 64)
    return k, v


SPLIT = [([131071], 1, 8, 2, 128, 128, "bf16"), ([131071], 1, 2, 1, 128, 64, "fp16"),
         ([70001], 5, 2, 1, 128, 128, "fp16"), ([40003], 3, 2, 1, 16, 64, "fp16"),
         ([50001, 33], 24, 4, 1, 64, 128, "fp16"), ([50001, 33], 24, 4, 1, 64, 128, "bf16"),
         ([20011, 0, 513], 160, 2, 2, 32, 64, "bf16"), ([60007], 6, 16, 2, 32, 64, "bf16")]


@pytest.mark.parametrize("lens,n,H,heads,bs,d,dtype", SPLIT)
def test_joined_means(lens, n, H, heads, bs, d, dtype):
    """Queries of zero: every visible key weighs 1, so O is the mean of their values and
    LSE the logarithm of their number. The weights are exact powers of two, so only
    O's own rounding and the fp32 sums are left: a share's, of at most 2^11 keys by MMAs
    of 16 (2^7 steps of 2^-23), and the join's over at most 2^9 shares, below 2^-12."""
    import torch
    rng = np.random.default_rng(n + d)
    need = [-(-x // bs) for x in lens]
    P = sum(need)
    k, v = keys_of(rng, P, heads, bs, d)
    cache = to_cache(k, v, np.full((P, heads), 2.0 ** -6), np.full((P, heads), 2.0 ** -7))
    ids = rng.permutation(P)
    table = np.zeros((len(lens), max(need)), dtype=np.int64)
    for b, m in enumerate(need):
        table[b, :m] = ids[sum(need[:b]):sum(need[:b]) + m]
    q = torch.zeros(len(lens) * n, H, d, device=DEV, dtype=tdt(dtype))
    o, lse = fa.attention_forward_cache(q, cache, ints(table), ints(lens),
                                        ints(np.arange(len(lens) + 1) * n))
    eps = torch.finfo(q.dtype).eps
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, L in enumerate(lens):
        for h in range(heads if L else 0):
            vv = U.CODE_VALUES[v[table[b, :need[b]], h]].reshape(-1, d)[:L] / 128.0
            total, size = np.cumsum(vv, 0), np.cumsum(np.abs(vv), 0)
            for i in range(n):
                lim = L - n + i + 1
                rows = got[b * n + i, h * (H // heads):(h + 1) * (H // heads)]
                if lim <= 0:
                    assert np.all(rows == 0)
                    continue
                ref, mag = total[lim - 1] / lim, size[lim - 1] / lim
                tol = 2.0 ** -12 * mag + np.abs(ref) * eps / 2 * (1 + 2.0 ** -10) + 2.0 ** -25
                assert np.all(np.abs(rows - ref) <= tol)
                le = gl[b * n + i, h * (H // heads):(h + 1) * (H // heads)]
                assert np.all(np.abs(le - np.log(lim)) <= 2.0 ** -12 + 2.0 ** -16)


@pytest.mark.parametrize("lens,n,H,heads,bs,d,dtype", SPLIT)
def test_joined_column_by_column(lens, n, H, heads, bs, d, dtype):
    """The same sizes with ordinary queries, every element against its own bound (the
    first two and the last two query tokens of each sequence)."""
    import torch
    rng = np.random.default_rng(n + d + 1)
    need = [-(-x // bs) for x in lens]
    P = sum(need)
    k, v = keys_of(rng, P, heads, bs, d)
    cache = to_cache(k, v, np.exp2(rng.integers(-8, -5, (P, heads))),
                     np.exp2(rng.integers(-9, -5, (P, heads))))
    ids = rng.permutation(P)
    table = np.zeros((len(lens), max(need)), dtype=np.int64)
    for b, m in enumerate(need):
        table[b, :m] = ids[sum(need[:b]):sum(need[:b]) + m]
    q = torch.from_numpy(rng.standard_normal((len(lens) * n, H, d))).to(DEV).to(tdt(dtype))
    o, lse = fa.attention_forward_cache(q, cache, ints(table), ints(lens),
                                        ints(np.arange(len(lens) + 1) * n))
    rows = n * (H // heads)
    floor = 2.0 ** -17 if d == 128 and 16 < rows <= 128 else 0.0
    host = [c.view(torch.uint8).cpu().numpy() for c in cache[:2]]
    scales = [s.double().cpu().numpy() for s in cache[2:]]
    eps = torch.finfo(q.dtype).eps
    for b, L in enumerate(lens):
        for i in sorted({0, 1, n - 2, n - 1} & set(range(n))):
            t = b * n + i
            lim = max(L - n + i + 1, 0)          # the keys that the causal rule leaves this token
            O, Ls, tol_o, tol_l = U.attend_columns(
                q[t:t + 1].double().cpu().numpy(), *host, *scales, table[b:b + 1], [lim], [0, 1], bs,
                d ** -0.5, False, eps, two_parts(rows, dtype), floor)
            got, gl = o[t].double().cpu().numpy(), lse[t].double().cpu().numpy()
            if lim == 0:
                assert np.all(got == 0) and np.all(np.isneginf(gl))
                continue
            err = np.abs(got - O[0])
            assert np.all(err <= tol_o[0]), f"O: {np.max(err / tol_o[0]):.2f} of the bound"
            assert np.all(np.abs(gl - Ls[0]) <= tol_l[0])


# ------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,H,heads,bs,d", [("bf16", 6, 2, 16, 64), ("fp16", 8, 1, 32, 128),
                                                ("bf16", 16, 2, 64, 128)])
def test_serving_loop_step_by_step(dtype, H, heads, bs, d):
    """Plan, append and attention as a serving loop makes them. Every step's plan is
    compared exactly, the codes and scales that its append leaves exactly, and its
    attention, element by element, with exact attention over those codes."""
    import torch
    rng = np.random.default_rng(d + bs)
    B, P, width = 4, 40, 12
    cache = fa.cache_empty(P, heads, bs, d, device=DEV)
    host = [np.zeros((P, heads, bs, d), np.uint8) for _ in range(2)]
    scales = [np.ones((P, heads)) for _ in range(2)]
    htable, hlens, hpos = np.full((B, width), -1, dtype=np.int64), [0] * B, 0
    hfree = rng.permutation(P)
    table, free, pos, lens = ints(htable), ints(hfree), ints([0]), ints(hlens)
    for add in ([37, 5, 64, 0], [1, 1, 1, 1], [1, 0, 2, 30], [3, 1, 1, 1], [1, 25, 1, 2], [1, 1, 1, 1]):
        T = sum(add)
        slots, cu, lens, pos = fa.cache_plan(lens, ints(add), table, free, pos, T, bs)
        hs, hcu, hlens, htable, hpos = U.plan(hlens, add, htable, hfree, hpos, T, bs)
        assert (slots.tolist(), cu.tolist(), lens.tolist(), pos.tolist()) == (hs, hcu, hlens, [hpos])
        assert np.array_equal(table.cpu().numpy(), htable)
        size = np.exp2(rng.integers(-3, 4, (T, heads, 1)))
        kv = [torch.from_numpy(rng.standard_normal((T, heads, d)) * size).to(DEV).to(tdt(dtype))
              for _ in range(2)]
        fa.cache_append(kv[0], kv[1], slots, cache)
        for i in range(2):
            host[i], scales[i] = U.append(kv[i].double().cpu().numpy(), hs, host[i], scales[i], bs)
            assert np.array_equal(cache[i].view(torch.uint8).cpu().numpy(), host[i])
            assert np.array_equal(cache[i + 2].cpu().numpy().astype(np.float64), scales[i])
        q = torch.from_numpy(rng.standard_normal((T, H, d))).to(DEV).to(tdt(dtype))
        rows = [n * (H // heads) for n in add]
        # (the wider of the bounds where a step's sequences go to different kernels)
        floor = 2.0 ** -17 if d == 128 and max(rows) > 16 else 0.0
        compare(q, cache, htable, hlens, hcu, True, None, dtype, two_parts(max(rows), dtype), floor)


# ------------------------------------------------------------ queries of wide range

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("top", [1.0, 60.0, 2.0 ** -10])
@pytest.mark.parametrize("n", [1, 3, 20, 40])
def test_elements_of_a_query_far_apart(n, top, dtype):
    """Elements of a query that lie 2^20 apart, 6 rows to the K / V head. Only where
    queries are cut into 8-bit parts (17 to 128 rows, on average 18 and 120 here, d 128)
    may small elements be rounded, by 2^-17 of the row's largest; with 6 rows, or 240,
    they count as they are."""
    import torch
    d, rng = 128, np.random.default_rng(n)
    apart = top * np.exp2(-np.linspace(0, 20, d)[rng.permutation(d)])
    cache = small_cache(rng, 40, 1, 32, d)
    lens, table = [n + 100, n, n + 259], rng.permutation(39).reshape(3, 13)
    q = torch.from_numpy(rng.standard_normal((3 * n, 6, d)) * apart).to(DEV).to(tdt(dtype))
    parts = 16 < 6 * n <= 128
    compare(q, cache, table, lens, [0, n, 2 * n, 3 * n], True, None, dtype, two_parts(6 * n, dtype),
            2.0 ** -17 if parts else 0.0)


# ------------------------------------------------------------ scores past fp32's whole numbers

@pytest.mark.parametrize("n,d", KERNELS)
@pytest.mark.parametrize("e", [18, 24, 27, 40])
def test_scores_of_any_size_choose_the_largest(n, d, e):
    """One key's score is 2^e (exponents whose fp32 steps are 2^(e - 23)) and the next
    one an eighth lower: O is the first key's V and LSE its score, to the rounding of
    the exponent: a weight that passes fp16's range is its largest number, 2^-5 less."""
    import torch
    rng = np.random.default_rng(e)
    P, bs = 10, 32
    k = np.zeros((P, 1, bs, d), np.uint8)
    k[:, 0, :, 0] = U.encode(rng.uniform(0.1, 0.875, (P, bs)))
    k[6, 0, 5, 0] = U.encode(np.array([1.0]))[0]
    v = U.encode(rng.standard_normal((P, 1, bs, d)))
    cache = to_cache(k, v, np.ones((P, 1)), np.full((P, 1), 0.37))
    q = torch.zeros(n, 1, d, device=DEV, dtype=torch.bfloat16)
    q[:, :, 0] = 2.0 ** e
    o, lse = fa.attention_forward_cache(q, cache, ints(np.arange(P)[None]), ints([P * bs]), ints([0, n]),
                                        False, 1.0)
    want = torch.from_numpy(U.CODE_VALUES[v[6, 0, 5]] * np.float64(np.float32(0.37))).to(DEV)
    assert ((o.double() - want).abs() <= want.abs() * 2.0 ** -5).all()
    assert ((lse.double() - 2.0 ** e).abs() <= 2.0 ** (e - 21)).all()


# ------------------------------------------------------------ a workspace of two graphs

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_two_graphs_on_one_workspace(dtype):
    """Two captured calls, one of single tokens and one of a mixture, that share a
    workspace and are replayed in turn on one stream give the bits of direct calls."""
    import torch
    rng = np.random.default_rng(3)
    cache = small_cache(rng, 120, 2, 32, 128)
    table, lens = ints(rng.permutation(120).reshape(3, 40)), ints([1270, 33, 900])
    cus = [ints([0, 1, 2, 3]), ints([0, 1, 61, 66])]
    qs = [torch.randn(T, 16, 128, device=DEV).to(tdt(dtype)) for T in (3, 66)]
    want = [fa.attention_forward_cache(q, cache, table, lens, cu) for q, cu in zip(qs, cus)]
    ws = torch.empty(max(fa.fa_fwd_cache_workspace_size(3, T, 16, 2, 128) for T in (3, 66)),
                     dtype=torch.uint8, device=DEV)
    outs = [(torch.empty_like(o), torch.empty_like(lse)) for o, lse in want]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in qs]
    for g, q, cu, (o, lse) in zip(graphs, qs, cus, outs):
        with torch.cuda.graph(g):
            fa.attention_forward_cache_into(q, cache, table, lens, o, lse, ws, cu)
    for _ in range(3):
        for o, lse in outs:
            o.zero_()
            lse.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
