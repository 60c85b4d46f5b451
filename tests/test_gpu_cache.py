"""The block cache on the GPU against the plain 64-bit implementations of
cache_util: planning (exact), appending (exact codes and scales) and attention
(bounds that count the roundings), over block sizes, head layouts, types,
lengths from zero on, ragged batches, bad blocks and hidden NaN; then the
three calls together, as a serving loop makes them."""
import numpy as np
import pytest

import attention_forward_flashattention_gb300 as fa
import cache_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    torch.cuda.init()
    fa.build.build()
    fa.load_library()


def ints(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def codes_of(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------ plan

def check_plan(lens, new, width, n_free, pos, T, bs, seed=0):
    rng = np.random.default_rng(seed)
    B = len(lens)
    table = rng.integers(0, 1 << 20, (B, width))
    free = rng.permutation(1 << 20)[:n_free]
    tab = ints(table)
    slots, cu, kv, nxt = fa.cache_plan(ints(lens), ints(new), tab, ints(free), ints([pos]), T, bs)
    ref = U.plan(list(map(int, lens)), list(map(int, new)), table, free, pos, T, bs)
    assert slots.tolist() == ref[0]
    assert cu.tolist() == ref[1] and kv.tolist() == ref[2] and nxt.tolist() == [ref[4]]
    assert np.array_equal(tab.cpu().numpy(), ref[3])


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("B,top,new", [(1, 0, 1), (1, 500, 300), (7, 100, 40), (33, 4000, 1),
                                       (513, 700, 9), (1500, 300, 20)])
def test_plan(B, top, new, bs):
    rng = np.random.default_rng(B + bs)
    lens, add = rng.integers(0, top + 1, B), rng.integers(0, new + 1, B)
    T = int(add.sum())
    check_plan(lens, add, (top + new) // bs + 2, T // bs + B + 5, 3, T + 3, bs)


@pytest.mark.parametrize("case", [
    dict(lens=[5, 0, 16, 15], new=[0, 0, 0, 0], T=0),            # nothing to do
    dict(lens=[5, 0, 16, 15], new=[0, 0, 0, 0], T=9),            # padding only
    dict(lens=[0, 3, 30, 2], new=[40, 20, 3, 14], n_free=3),     # blocks run out
    dict(lens=[0, 3, 30, 2], new=[40, 20, 3, 14], n_free=0),
    dict(lens=[0, 3, 30, 2], new=[40, 20, 3, 14], pos=99),       # free_pos out of range
    dict(lens=[0, 3, 30, 2], new=[40, 20, 3, 14], pos=-1),
    dict(lens=[0, 3, 30, 2], new=[40, 20, 3, 14], T=70),         # rows run out
    dict(lens=[-4, 3, 30, 2], new=[40, -20, 3, 14]),             # negative numbers
    dict(lens=[0, 2 ** 31 - 1, 5], new=[3, 2 ** 31 - 1, 4]),     # sums past 32 bits
    dict(lens=[2 ** 31 - 1] * 3, new=[2 ** 31 - 1] * 3, T=50),
    dict(lens=[0, 100, 2], new=[1, 60, 1], width=9),             # table row too short
])
def test_plan_refusals(case):
    c = {**dict(width=12, n_free=20, pos=0), **case}
    T = c.get("T", sum(m for m in c["new"] if 0 < m < 1000))
    check_plan(c["lens"], c["new"], c["width"], c["n_free"], c["pos"], T, 16)


def test_plan_bad_table_entry_gives_no_slot():
    tab = ints([[-1, 5], [1 << 27, 5]])
    slots, _, kv, _ = fa.cache_plan(ints([3, 3]), ints([2, 2]), tab, ints([9]), ints([0]), 4, 16)
    assert slots.tolist() == [-1] * 4 and kv.tolist() == [5, 5]


# ------------------------------------------------------------ append

def make_cache(P, heads, bs, d, layout, rng, fill=True):
    """A cache (contiguous, token-major, or K and V side by side) of random
    codes without NaN, and power-of-two scales."""
    import torch
    if layout == "head":
        k, v = (torch.zeros(P, heads, bs, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    elif layout == "token":
        k, v = (torch.zeros(P, bs, heads, d, dtype=torch.uint8, device=DEV).transpose(1, 2)
                for _ in range(2))
    else:   # one storage [P, 2, heads, bs, d + 16]
        s = torch.zeros(P, 2, heads, bs, d + 16, dtype=torch.uint8, device=DEV)
        k, v = s[:, 0, :, :, :d], s[:, 1, :, :, :d]
    if fill:
        for t in (k, v):
            c = rng.integers(0, 256, (P, heads, bs, d), dtype=np.uint8)
            t.copy_(torch.from_numpy(np.where((c & 0x7F) == 0x7F, c ^ 1, c).astype(np.uint8)))
    ks, vs = (torch.from_numpy(np.exp2(rng.integers(-9, -3, (P, heads))).astype(np.float32)).to(DEV)
              for _ in range(2))
    return fa.Cache(k, v, ks, vs)


def tdt(name):
    import torch
    return torch.float16 if name == "fp16" else torch.bfloat16


def slots_of(runs):
    return [s0 + i for s0, n in runs for i in range(n)]


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,heads,layout", [("fp16", 1, "head"), ("bf16", 3, "token"),
                                                ("fp16", 5, "pair")])
def test_append(bs, d, dtype, heads, layout):
    import torch
    rng = np.random.default_rng(bs + d + heads)
    P = 24
    cache = make_cache(P, heads, bs, d, layout, rng)
    pages = rng.permutation(P)
    # single tokens into partly filled blocks, one that starts a block, a whole
    # block, one that ends and continues in another, padding in between
    runs = [(pages[0] * bs + 3, 1), (pages[1] * bs + bs - 1, 1), (pages[2] * bs, 1), (-1, 1),
            (pages[3] * bs, bs), (pages[4] * bs + 5, bs - 5), (pages[5] * bs, 7),
            (pages[6] * bs + 1, bs - 2), (-5, 1), (P * bs, 1), (pages[7] * bs + 2, 2),
            (pages[8] * bs, bs), (pages[9] * bs, bs), (pages[10] * bs, bs - 1)]
    slots = slots_of(runs)
    T = len(slots)
    size = np.exp2(rng.integers(-6, 9, (T, heads, 1)))   # scales grow in some blocks
    x = [torch.from_numpy(rng.standard_normal((T, heads, d)) * size).to(DEV).to(tdt(dtype))
         for _ in range(2)]
    x[0][4, 0, 1], x[0][4, 0, 5], x[1][5, 0, 2] = float("inf"), float("nan"), -float("inf")
    x[1][7, :, :] = 0
    before = [codes_of(cache.k), codes_of(cache.v), cache.k_scales.cpu().numpy(),
              cache.v_scales.cpu().numpy()]
    fa.cache_append(x[0], x[1], ints(slots), cache)
    for i, (t, s) in enumerate(((cache.k, cache.k_scales), (cache.v, cache.v_scales))):
        want, ws = U.append(x[i].double().cpu().numpy(), slots, before[i], before[i + 2], bs)
        got = codes_of(t)
        assert np.array_equal(s.cpu().numpy().astype(np.float64), ws)
        nan = (want & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan)
        assert np.array_equal(got[~nan], want[~nan])


def test_append_many_tokens_ragged():
    """Runs that cross every tile border, on strided inputs."""
    import torch
    rng = np.random.default_rng(5)
    bs, heads, d = 64, 2, 128
    sizes = rng.integers(1, 150, 40)
    offs = rng.integers(0, bs, 40)
    P = int(sum((o + n + bs - 1) // bs for o, n in zip(offs, sizes)))
    cache = make_cache(P, heads, bs, d, "head", rng)
    slots, page = [], 0
    for o, n in zip(offs, sizes):
        slots += [page * bs + o + i for i in range(n)]
        page += (o + n + bs - 1) // bs
    T = len(slots)
    store = torch.randn(T, 3, heads, d, device=DEV).to(torch.bfloat16)
    k, v = store[:, 0], store[:, 2]
    before = [codes_of(cache.k), codes_of(cache.v), cache.k_scales.cpu().numpy(),
              cache.v_scales.cpu().numpy()]
    fa.cache_append(k, v, ints(slots), cache)
    for i, (x, t, s) in enumerate(((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales))):
        want, ws = U.append(x.double().cpu().numpy(), slots, before[i], before[i + 2], bs)
        assert np.array_equal(codes_of(t), want)
        assert np.array_equal(s.cpu().numpy().astype(np.float64), ws)


def test_append_old_scale_that_is_no_power_of_two():
    """It is rounded up to one, and the older codes follow: within half a code
    step (2^-4) of their values, twice rounded."""
    import torch
    rng = np.random.default_rng(6)
    cache = make_cache(2, 1, 16, 64, "head", rng)
    cache.k_scales[1, 0] = 0.3
    old = U.CODE_VALUES[codes_of(cache.k)[1, 0, :4]] * float(np.float32(0.3))
    x = torch.ones(1, 1, 64, dtype=torch.float16, device=DEV)
    fa.cache_append(x, x, ints([20]), cache)
    assert cache.k_scales[1, 0].item() == 0.5
    new = U.CODE_VALUES[codes_of(cache.k)[1, 0, :5]] * 0.5
    assert np.all(np.abs(new[:4] - old) <= 2.0 ** -4 * np.abs(old) + 2.0 ** -10 * 0.5)
    assert np.all(new[4] == 1.0)


# ------------------------------------------------------------ attention

def attention_case(lens, counts, H, heads, bs, d, dtype, causal, layout="head", uniform=False,
                   seed=0, spoil=None, scale=None, q_mult=1.0, width=None, q_layout="thd",
                   q_floor=0.0):
    """Runs fa_fwd_cache and compares it with the 64-bit implementation.
    spoil(k codes, v codes, table): changes what the call must not see. q_floor:
    rounding of a query element, relative to the largest one of its row."""
    import torch
    rng = np.random.default_rng(seed)
    B = len(lens)
    need = [(max(x, 0) + bs - 1) // bs for x in lens]
    P = sum(need) + 3
    cache = make_cache(P, heads, bs, d, layout, rng)
    width = max(1, max(need)) if width is None else width
    table = np.full((B, width), -1, dtype=np.int64)
    ids = rng.permutation(P)
    at = 0
    for b, n in enumerate(need):
        table[b, :min(n, width)] = ids[at:at + min(n, width)]
        at += n
    cu = np.concatenate([[0], np.cumsum(counts)])
    T = int(cu[-1])
    q = torch.from_numpy(rng.standard_normal((T, H, d)) * q_mult).to(DEV).to(tdt(dtype))
    qv = q.double().cpu().numpy()
    ks, vs = cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy()
    scale = d ** -0.5 if scale is None else scale
    ref = U.attend(qv, codes_of(cache.k), codes_of(cache.v), ks.astype(np.float64),
                   vs.astype(np.float64), table, lens, cu, bs, scale, causal)
    if q_floor:   # of a score: q_floor max |q| sum |k|
        most = (np.abs(U.CODE_VALUES[codes_of(cache.k)]).sum(-1) * ks[:, :, None]).max()
        far = ref[3] + scale * q_floor * np.abs(qv).max(-1) * most
        ref = (ref[0], ref[1], ref[2], far, ref[4])
    if spoil is not None:
        spoil(cache, table, ids[at:])
    if uniform:
        n = counts[0]
        q4 = q.reshape(B, n, H, d).transpose(1, 2)
        if q_layout == "bhnd":
            q4 = q4.contiguous()
        o, lse = fa.attention_forward_cache(q4, cache, ints(table), ints(lens), None, causal, scale)
        assert o.shape == q4.shape and lse.shape == q4.shape[:-1]
        o, lse = o.transpose(1, 2).reshape(T, H, d), lse.transpose(1, 2).reshape(T, H)
    else:
        o, lse = fa.attention_forward_cache(q, cache, ints(table), ints(lens), ints(cu), causal,
                                            scale)
    assert fa.fa_check(0) == fa.FA_OK
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    eps = torch.finfo(tdt(dtype)).eps
    tol_o, tol_l = U.attend_tolerance(ref, eps, max(1, max(lens)))
    empty = np.isneginf(ref[1])
    assert np.array_equal(np.isneginf(gl), empty) and np.all(got[empty] == 0)
    err, le = np.abs(got - ref[0]), np.abs(gl[~empty] - ref[1][~empty])
    assert np.all(np.isfinite(got)), "not finite"
    assert np.all(err <= tol_o), f"O: {err.max():.2e}, {np.max(err / tol_o):.2f} of the bound"
    assert np.all(le <= tol_l[~empty]), f"LSE: {np.max(le / tol_l[~empty]):.2f} of the bound"


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("d,dtype,H,heads", [(64, "fp16", 4, 4), (128, "bf16", 6, 2),
                                             (128, "fp16", 8, 1), (64, "bf16", 3, 1)])
def test_single_tokens(bs, d, dtype, H, heads):
    lens = [1, 0, bs, bs + 1, 300, 17, 2 * bs - 1, 641]
    attention_case(lens, [1] * len(lens), H, heads, bs, d, dtype, True, seed=bs)


@pytest.mark.parametrize("layout", ["token", "pair"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,dtype,H,heads,bs", [(64, "fp16", 4, 2, 16), (128, "bf16", 4, 4, 64),
                                                (128, "fp16", 20, 2, 128)])
def test_ragged_queries(layout, causal, d, dtype, H, heads, bs):
    lens = [200, 5, 0, 129, 77, 400]
    counts = [3, 5, 2, 1, 0, 40]      # among them a row longer than nothing, and no row at all
    attention_case(lens, counts, H, heads, bs, d, dtype, causal, layout)


@pytest.mark.parametrize("n,H,heads", [(1, 32, 1), (2, 24, 8), (4, 4, 4), (5, 8, 1), (9, 4, 2),
                                       (17, 8, 8), (64, 2, 1), (130, 6, 2)])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_query_counts(n, H, heads, d, dtype):
    attention_case([n, n + 133, 260], [n] * 3, H, heads, 32, d, dtype, True, uniform=True,
                   q_layout="bhnd" if n % 2 else "bnhd", seed=n)


@pytest.mark.parametrize("d,dtype,H,heads,bs", [(128, "bf16", 8, 2, 64), (64, "fp16", 16, 4, 16),
                                                (128, "fp16", 2, 2, 128), (64, "bf16", 60, 1, 32)])
def test_mixed_batches(d, dtype, H, heads, bs):
    """Single tokens, drafts and chunks in one call, with and without room for them."""
    lens = [700, 33, 1, 0, 260, 900, 64, 130, 5, 1024]
    counts = [1, 1, 1, 1, 200, 7, 0, 130, 3, 1]
    attention_case(lens, counts, H, heads, bs, d, dtype, True, seed=d + H)
    attention_case(lens, counts[::-1], H, heads, bs, d, dtype, False, seed=d + H + 1)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("d,dtype", [(128, "fp16"), (64, "bf16")])
def test_mixed_batches_of_few_rows(group, d, dtype):
    """Pieces of every number of rows around 8 and 16 beside a chunk."""
    counts = sorted({n for r in (1, 7, 8, 9, 15, 16, 17) for n in (r // group, -(-r // group)) if n})
    lens = [40 * n + 3 for n in counts] + [170, 0]
    attention_case(lens, counts + [150, 1], 2 * group, 2, 32, d, dtype, True, seed=group)


@pytest.mark.parametrize("lens,counts", [([3, 0, 40], [10, 1, 45]), ([1], [300])])
def test_rows_before_the_first_key(lens, counts):
    """More query rows than keys: the first rows see nothing."""
    attention_case(lens, counts, 4, 2, 16, 64, "fp16", True)
    attention_case(lens, counts, 2, 2, 16, 128, "bf16", True)


@pytest.mark.parametrize("n,H,heads", [(1, 8, 2), (6, 8, 1), (140, 2, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_and_blocks_out_of_sight(n, H, heads, d):
    """NaN behind the last key, in blocks of other sequences, in scales of
    unused blocks; and, for the causal rule, keys that later rows alone see."""
    def spoil(cache, table, unused):
        for b, x in enumerate((n + 50, n, n + 200)):
            last = table[b, (x - 1) // 32]
            if x % 32:
                cache.k.view_as(cache.k)[int(last), :, x % 32:] = 0x7F
                cache.v[int(last), :, x % 32:] = 0xFF
        for u in unused:
            cache.k_scales[int(u)] = float("nan")
            cache.v_scales[int(u)] = float("nan")
    attention_case([n + 50, n, n + 200], [n] * 3, H, heads, 32, d, "fp16", True, spoil=spoil)


@pytest.mark.parametrize("n,H", [(3, 2), (20, 4), (20, 8), (150, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_reaches_the_rows_that_see_it(n, H, d):
    """A key whose V holds NaN in one column: the rows that see the key get NaN
    there and nowhere else, earlier rows get finite values."""
    import torch
    rng = np.random.default_rng(3)
    L, bs = n + 70, 16
    P = (L + bs - 1) // bs
    cache = make_cache(P, 1, bs, d, "head", rng)
    table = rng.permutation(P)[None]
    q = torch.randn(n, H, d, device=DEV).to(torch.bfloat16)
    clean, cl = fa.attention_forward_cache(q, cache, ints(table), ints([L]), ints([0, n]))
    first = n // 2                            # the first row that sees the key
    j = L - n + first
    cache.v[int(table[0, j // bs]), 0, j % bs, 37] = 0x7F
    o, lse = fa.attention_forward_cache(q, cache, ints(table), ints([L]), ints([0, n]))
    assert torch.equal(lse, cl)
    nan = torch.isnan(o)
    assert nan[first:, :, 37].all() and int(nan.sum()) == (n - first) * H
    assert torch.equal(o[~nan], clean[~nan])


def test_bad_blocks_hide_their_keys():
    import torch
    rng = np.random.default_rng(8)
    for n, H, d in ((1, 4, 64), (3, 16, 128), (140, 2, 128)):
        lens, bs = [n + 90, n + 20], 16
        P = 40
        cache = make_cache(P, 2, bs, d, "head", rng)
        table = rng.permutation(P)[:20].reshape(2, 10)
        if n > 100:
            table = rng.permutation(P)[:32].reshape(2, 16)
        table[0, 2], table[1, 0], table[0, 4] = -7, P, 2 ** 31 - 1
        q = torch.randn(2 * n, H, d, device=DEV).to(torch.float16)
        cu = [0, n, 2 * n]
        o, lse = fa.attention_forward_cache(q, cache, ints(table), ints(lens), ints(cu))
        ref = U.attend(q.double().cpu().numpy(), codes_of(cache.k), codes_of(cache.v),
                       cache.k_scales.double().cpu().numpy(), cache.v_scales.double().cpu().numpy(),
                       table, lens, cu, bs, d ** -0.5, True)
        tol_o, tol_l = U.attend_tolerance(ref, 2.0 ** -10, max(lens))
        assert np.all(np.abs(o.double().cpu().numpy() - ref[0]) <= tol_o)
        seen = np.isfinite(ref[1])
        gl = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(gl), ~seen)
        assert np.all(np.abs(gl - ref[1])[seen] <= tol_l[seen])
        # all blocks bad: nothing is seen
        o, lse = fa.attention_forward_cache(q, cache, ints(np.full_like(table, -1)), ints(lens),
                                            ints(cu))
        assert (o == 0).all() and torch.isneginf(lse).all()


def test_lengths_out_of_range_are_clamped():
    import torch
    rng = np.random.default_rng(9)
    cache = make_cache(8, 1, 16, 64, "head", rng)
    table = ints(np.arange(8).reshape(2, 4))
    q = torch.randn(2, 1, 64, device=DEV).to(torch.float16)
    a = fa.attention_forward_cache(q, cache, table, ints([64, 0]))
    b = fa.attention_forward_cache(q, cache, table, ints([2 ** 31 - 1, -5]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_of_no_sequence_are_left_alone():
    """Rows before the first sequence's and behind the last one's, and offsets
    out of range."""
    import torch
    rng = np.random.default_rng(10)
    cache = make_cache(8, 2, 16, 64, "head", rng)
    table, lens = ints(np.arange(8).reshape(2, 4)), ints([30, 50])
    q = torch.randn(9, 4, 64, device=DEV).to(torch.float16)
    ws = torch.empty(fa.fa_fwd_cache_workspace_size(2, 9, 4, 2, 64), dtype=torch.uint8, device=DEV)

    def run(cu):
        o = torch.full_like(q, 7.0)
        lse = torch.full((9, 4), 7.0, device=DEV)
        fa.attention_forward_cache_into(q, cache, table, lens, o, lse, ws, ints(cu))
        return o, lse
    o, lse = run([1, 3, 6])
    full, fl = fa.attention_forward_cache(q[1:6], cache, table, lens, ints([0, 2, 5]))
    assert torch.equal(o[1:6], full) and torch.equal(lse[1:6], fl)
    for r in (0, 6, 7, 8):
        assert (o[r] == 7).all() and (lse[r] == 7).all()
    o, lse = run([5, 2, 2 ** 31 - 1])      # the first sequence has no rows, the second seven
    assert (o[:2] == 7).all() and not (o[2:] == 7).all(dim=-1).any()


def test_wide_values_and_scales():
    """Sharp rows, V scales far apart, and 16-bit extremes of q."""
    import torch
    attention_case([700, 300], [1, 1], 4, 2, 16, 128, "bf16", True, q_mult=8.0)
    attention_case([700, 300], [33, 40], 4, 2, 16, 64, "fp16", True, q_mult=8.0)
    rng = np.random.default_rng(11)
    for n, dtype, qs in ((1, "bf16", 2.0 ** 40), (20, "bf16", 2.0 ** 40), (1, "fp16", 60.0),
                         (20, "bf16", 2.0 ** -100), (150, "bf16", 2.0 ** 40)):
        lens, bs, H, d = [n + 100], 16, 2, 64
        P = (lens[0] + bs - 1) // bs
        cache = make_cache(P, 1, bs, d, "head", rng)
        cache.v_scales.copy_(torch.from_numpy(np.exp2(rng.integers(-40, 40, (P, 1)))).to(DEV))
        cache.k_scales.mul_(2.0 ** -40 if qs > 1e9 else 1.0)
        table = rng.permutation(P)[None]
        q = (torch.randn(n, H, d, device=DEV) * qs).to(tdt(dtype))
        o, lse = fa.attention_forward_cache(q, cache, ints(table), ints(lens), ints([0, n]))
        ref = U.attend(q.double().cpu().numpy(), codes_of(cache.k), codes_of(cache.v),
                       cache.k_scales.double().cpu().numpy(), cache.v_scales.double().cpu().numpy(),
                       table, lens, [0, n], bs, d ** -0.5, True)
        tol_o, tol_l = U.attend_tolerance(ref, torch.finfo(tdt(dtype)).eps, lens[0])
        got = o.double().cpu().numpy()
        if dtype == "fp16":   # results above its range are infinite
            fine = np.abs(ref[0]) < 60000
            assert np.all(np.abs(got - ref[0])[fine] <= tol_o[fine])
        else:
            assert np.all(np.abs(got - ref[0]) <= tol_o)
        assert np.all(np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_l)


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
def test_up_to_128_rows_on_average(bs, dtype, causal):
    """Drafts beside pieces of more rows than one item holds, single tokens and
    sequences without rows, 68 rows of a K / V head on average."""
    lens = [900, 127, 0, 300, 64, 1290, 5, 33]
    counts = [70, 5, 2, 33, 0, 17, 1, 8]
    attention_case(lens, counts, 8, 2, bs, 128, dtype, causal, seed=bs)
    attention_case([400, 129, 31], [20, 20, 20], 6, 1, bs, 128, dtype, causal, uniform=True,
                   seed=bs + 1)
    attention_case([0, 60, 0, 7, 200], [20, 20, 33, 30, 25], 2, 2, bs, 128, dtype, causal, seed=bs + 2)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,top", [(20, 1.0), (20, 60.0), (20, 2.0 ** -12), (150, 60.0), (3, 60.0)])
def test_queries_of_wide_range(dtype, n, top):
    """Elements of a query that lie 2^20 apart: the small ones may be rounded to
    2^-17 of the largest (half of the last part's smallest step, 2^-10, of a row
    whose largest element is at least 2^7)."""
    mult = top * np.exp2(-np.linspace(0, 20, 128)[np.random.default_rng(n).permutation(128)])
    attention_case([n + 100, n, n + 259], [n] * 3, 6, 1, 32, 128, dtype, True, q_mult=mult,
                   q_floor=2.0 ** -17)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,d,keys", [(24, 128, 253), (12, 64, 253), (24, 64, 253), (150, 128, 253),
                                      (12, 128, 6000), (24, 128, 6000), (150, 128, 6000)])
def test_queries_without_a_value(dtype, n, d, keys):
    """Zero rows see the mean of V; rows with an infinity or NaN give NaN, and the
    others are what they are without them."""
    import torch
    rng = np.random.default_rng(5)
    H, bs = 2, 32
    P = -(-keys // bs)
    cache = make_cache(P, 2 if n == 12 else 1, bs, d, "head", rng)
    table, lens = ints(rng.permutation(P)[None]), ints([keys])
    q = torch.from_numpy(rng.standard_normal((n, H, d))).to(DEV).to(tdt(dtype))
    clean, cl = fa.attention_forward_cache(q, cache, table, lens, ints([0, n]))
    q[3] = 0
    q[7, 0, 5], q[9, 1, 40], q[11, 0, d - 1] = float("inf"), float("nan"), -float("inf")
    o, lse = fa.attention_forward_cache(q, cache, table, lens, ints([0, n]))
    bad = torch.zeros(n, H, dtype=torch.bool, device=DEV)
    bad[7, 0] = bad[9, 1] = bad[11, 0] = True
    assert torch.isnan(o[bad]).all() and not torch.isfinite(lse[bad]).any()
    good = ~bad
    good[3] = False
    assert torch.equal(o[good], clean[good]) and torch.equal(lse[good], cl[good])
    seen = keys - n + 4
    want = np.log(seen)
    most = seen * 2.0 ** -24 + 2.0 ** -20 + 8 * 2.0 ** -24 * (want + 64)   # (attend_tolerance's)
    assert np.all(np.abs(lse[3].cpu().numpy() - want) <= most)


def test_long_sequences_split_and_joined():
    """Few rows over many keys: the work of a row is shared and joined. Against
    a float64 evaluation on the GPU."""
    import torch
    rng = np.random.default_rng(12)
    for lens, n, H, heads, bs, d, dtype in (
            ([131071, 1, 70000], 1, 8, 2, 128, 128, "bf16"), ([40003], 3, 2, 1, 16, 64, "fp16"),
            ([50001, 33], 24, 4, 1, 64, 128, "fp16"), ([30011, 0, 513], 160, 2, 2, 32, 64, "bf16"),
            ([70001], 5, 8, 1, 128, 128, "bf16"), ([70001], 3, 8, 1, 16, 128, "fp16"),
            ([60007], 6, 16, 2, 32, 64, "bf16")):
        B = len(lens)
        need = [(x + bs - 1) // bs for x in lens]
        P = sum(need)
        cache = make_cache(P, heads, bs, d, "head", rng)
        table = np.zeros((B, max(need)), dtype=np.int64)
        ids, at = rng.permutation(P), 0
        for b, m in enumerate(need):
            table[b, :m] = ids[at:at + m]
            at += m
        q = torch.randn(B * n, H, d, device=DEV).to(tdt(dtype))
        cu = np.arange(B + 1) * n
        o, lse = fa.attention_forward_cache(q, cache, ints(table), ints(lens), ints(cu))
        vals = torch.from_numpy(U.CODE_VALUES).to(DEV)
        for b, L in enumerate(lens):
            for h in range(heads if L else 0):
                rows = torch.from_numpy(table[b, :need[b]]).to(DEV)
                kk, vv = ((vals[c.view(torch.uint8)[rows, h].long()]
                           * s[rows, h].double()[:, None, None]).reshape(-1, d)[:L]
                          for c, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)))
                for i in range(n):
                    lim = L - n + i + 1
                    qq = q[b * n + i, h * (H // heads):(h + 1) * (H // heads)].double()
                    if lim <= 0:
                        assert (o[b * n + i] == 0).all()
                        continue
                    s = qq @ kk[:lim].T * d ** -0.5
                    ref_l = torch.logsumexp(s, -1)
                    p = torch.exp(s - ref_l[:, None])
                    ref_o, mag = p @ vv[:lim], p @ vv[:lim].abs()
                    sl = slice(h * (H // heads), (h + 1) * (H // heads))
                    got = o[b * n + i, sl].double()
                    far = ((d + 3) * 2.0 ** -24 * d ** -0.5
                           * (qq.abs() @ kk[:lim].abs().T).amax())
                    # fp32 sums run over at most 8192 keys before they are joined
                    rel = 2.0 ** -11 + 2 * far + 2.0 ** -11 + 2.0 ** -20
                    eps = torch.finfo(q.dtype).eps
                    small = 2.0 ** -25 * 448 * lim * float(cache.v_scales.max())
                    assert ((got - ref_o).abs() <= mag * rel + ref_o.abs() * eps / 2 + small).all()
                    assert ((lse[b * n + i, sl].double() - ref_l).abs()
                            <= far + 2.0 ** -11 + 2.0 ** -16).all()


def test_cache_past_32_bits():
    """Blocks whose byte offsets pass 2^32: rows at the far end of a large
    cache, written and read."""
    import torch
    bs, heads, d = 128, 16, 128
    P = (5 << 30) // (heads * bs * d) + 1          # more than 5 GB of K, and of V
    k, v = (torch.empty(P, heads, bs, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.ones(P, heads, device=DEV) for _ in range(2))
    cache = fa.Cache(k, v, ks, vs)
    x, y = (torch.randn(200, heads, d, device=DEV).to(torch.bfloat16) for _ in range(2))
    table = ints([[P - 1, P // 2]])
    slots, cu, kv, _ = fa.cache_plan(ints([0]), ints([200]), ints([[-1, -1]]), ints([P - 1, P // 2]),
                                     ints([0]), 200, bs)
    fa.cache_append(x, y, slots, cache)
    small = fa.cache_empty(2, heads, bs, d, device=DEV)
    fa.cache_append(x, y, ints(np.arange(200)), small)
    assert torch.equal(k[P - 1], small.k[0].view(torch.uint8))
    assert torch.equal(v[P // 2, :, :72], small.v[1, :, :72].view(torch.uint8))
    q = torch.randn(1, heads, d, device=DEV).to(torch.bfloat16)
    a = fa.attention_forward_cache(q, cache, table, kv)
    b = fa.attention_forward_cache(q, small, ints([[0, 1]]), kv)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    q = torch.randn(200, heads, d, device=DEV).to(torch.bfloat16)
    a = fa.attention_forward_cache(q, cache, table, kv, cu)
    b = fa.attention_forward_cache(q, small, ints([[0, 1]]), kv, cu)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


# ------------------------------------------------------------ together

def serve(stream=None, steps=6, seed=1):
    """A small serving loop: prompts of different lengths, then single tokens.
    Returns each step's (o, lse) and the keys and values appended."""
    import torch
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, H, heads, bs, d = 3, 6, 2, 16, 64
    cache = fa.cache_empty(40, heads, bs, d, device=DEV)
    table = ints(np.full((B, 12), -1))
    free, pos, lens = ints(np.random.default_rng(seed).permutation(40)), ints([0]), ints([0] * B)
    out, hist = [], [[] for _ in range(B)]
    adds = [[37, 5, 64]] + [[1, 1, 1], [1, 0, 2], [1, 1, 1], [3, 1, 1], [1, 1, 1]][:steps - 1]
    for add in adds:
        T = sum(add)
        slots, cu, lens, pos = fa.cache_plan(lens, ints(add), table, free, pos, T, bs, stream)
        q = torch.randn(T, H, d, device=DEV, generator=g).to(torch.bfloat16)
        k, v = (torch.randn(T, heads, d, device=DEV, generator=g).to(torch.bfloat16)
                for _ in range(2))
        fa.cache_append(k, v, slots, cache, stream)
        out.append((q, add) + fa.attention_forward_cache(q, cache, table, lens, cu, stream=stream))
        at = 0
        for b, n in enumerate(add):
            hist[b].append((k[at:at + n], v[at:at + n]))
            at += n
    return out, hist, cache


def test_serving_loop():
    """Plan, append and attention as a serving loop: each step's attention
    against exact attention over the 16-bit keys and values appended so far.
    An 8-bit code is within 2^-4 of its value, relatively, or half the
    smallest code step of its block's scale (2^-10 of it), and once more by
    2^-4 where a grown scale rounded it again below the normal codes; so
    scores move by at most scale sum |q| |dk|, and O by the weighted |dv| plus
    the change of the weights."""
    import torch
    out, hist, cache = serve()
    torch.cuda.synchronize()
    steps = len(out)
    for t in range(steps):
        q, add, o, lse = out[t]
        at = 0
        for b, n in enumerate(add):
            k = torch.cat([x[0] for x in hist[b][:t + 1]]).double()
            v = torch.cat([x[1] for x in hist[b][:t + 1]]).double()
            for i in range(n):
                lim = len(k) - n + i + 1
                for h in range(6):
                    kk, vv = k[:lim, h // 3], v[:lim, h // 3]
                    qq = q[at + i, h].double()
                    s = kk @ qq / 8.0
                    # largest scale: amax < 8 for these normal values, so s <= 2^-5
                    dk = kk.abs() * 2.0 ** -4 + 2.0 ** -15 * 2
                    ds = (dk @ qq.abs()).max() / 8.0
                    p = torch.softmax(s, 0)
                    dv = vv.abs() * 2.0 ** -4 + 2.0 ** -15 * 2
                    bound = p @ dv + 2 * torch.expm1(ds) * (p @ (vv.abs() + dv)) + 2.0 ** -8 * 8
                    assert ((o[at + i, h].double() - p @ vv).abs() <= bound).all()
                    assert abs(lse[at + i, h].double() - torch.logsumexp(s, 0)) <= ds + 1e-3
            at += n


def test_serving_loop_on_streams_and_twice():
    """The same loop on two streams at once gives the same bits."""
    import torch
    ref, _, c0 = serve()
    torch.cuda.synchronize()
    main = torch.cuda.current_stream()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(main)
        with torch.cuda.stream(s):
            got.append(serve(s))
    torch.cuda.synchronize()
    for out, _, c in got:
        for a, b in zip(ref, out):
            assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
        assert torch.equal(c.k.view(torch.uint8), c0.k.view(torch.uint8))
        assert torch.equal(c.v_scales, c0.v_scales)


@pytest.mark.parametrize("n,H,heads,d", [(1, 8, 2, 128), (40, 4, 1, 64), (5, 16, 2, 128)])
def test_graph_replays_a_step(n, H, heads, d):
    """One step captured (plan, append, attention), replayed on new lengths and
    values, against direct calls."""
    import torch
    rng = np.random.default_rng(n)
    B, bs = 4, 32
    P = 64
    base = make_cache(P, heads, bs, d, "head", rng)
    st = dict(lens=ints([0] * B), new=ints([n] * B), table=ints(np.arange(B * 12).reshape(B, 12)),
              free=ints(np.arange(48, 64)), pos=ints([0]))
    x = [torch.empty(B * n, heads, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    q = torch.empty(B * n, H, d, dtype=torch.bfloat16, device=DEV)
    cap = fa.Cache(*(t.clone() for t in base))

    def step(c, table):
        slots, cu, kv, nxt = fa.cache_plan(st["lens"], st["new"], table, st["free"], st["pos"],
                                           B * n, bs)
        fa.cache_append(x[0], x[1], slots, c)
        return fa.attention_forward_cache(q, c, table, kv, cu) + (nxt,)

    def fill(seed):
        r = np.random.default_rng(seed)
        st["lens"].copy_(ints(r.integers(1, 200, B)))
        for t in (*x, q):
            t.copy_(torch.from_numpy(r.standard_normal(t.shape)).to(DEV))
        st["table"].copy_(ints(np.arange(B * 12).reshape(B, 12)))
        for a, b in zip(cap, base):
            a.copy_(b)

    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cap, st["table"])
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(cap, st["table"])
    for seed in (1, 2, 3):
        fill(seed)
        c2, t2 = fa.Cache(*(t.clone() for t in base)), st["table"].clone()
        want = step(c2, t2)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(st["table"], t2)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cap, c2))
    assert fa.fa_check(0) == fa.FA_OK


def test_workspace_and_empty_calls():
    """A workspace that is too small is refused; calls of nothing succeed."""
    import torch
    rng = np.random.default_rng(20)
    cache = make_cache(4, 2, 16, 64, "head", rng)
    tab, lens = ints(np.arange(4).reshape(2, 2)), ints([20, 30])
    q = torch.randn(2, 4, 64, device=DEV).half()
    o, lse = torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device=DEV)
    size = fa.fa_fwd_cache_workspace_size(2, 2, 4, 2, 64)
    with pytest.raises(fa.FaError) as e:
        fa.attention_forward_cache_into(q, cache, tab, lens, o, lse,
                                        torch.empty(size - 16, dtype=torch.uint8, device=DEV))
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (o == 7).all() and (lse == 7).all()
    fa.attention_forward_cache_into(q, cache, tab, lens, o, lse,
                                    torch.empty(size, dtype=torch.uint8, device=DEV))
    assert not (o == 7).all()
    desc = fa.FaCache(cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scales.data_ptr(),
                      cache.v_scales.data_ptr(), 4, 16, 2, 64, 2 * 16 * 64, 16 * 64, 64)
    st = ((8, 64, 128), (8, 64, 128))
    assert fa.fa_cache_append(q.data_ptr(), q.data_ptr(), st, lens.data_ptr(), 0, desc,
                              fa.FA_DTYPE_FP16) == fa.FA_OK
    assert fa.fa_fwd_cache(q.data_ptr(), desc, tab.data_ptr(), 2, lens.data_ptr(), None,
                           o.data_ptr(), lse.data_ptr(), 2, 0, 4, st, True, 0.1, fa.FA_DTYPE_FP16,
                           o.data_ptr(), 0) in (fa.FA_OK, fa.FA_ERR_INVALID_ARG)
    slots, cu, kv, nxt = fa.cache_plan(ints([3]), ints([0]), ints([[1]]), ints([]), ints([0]), 0, 16)
    assert slots.numel() == 0 and cu.tolist() == [0, 0] and kv.tolist() == [3] and nxt.tolist() == [0]


def test_concurrent_calls_on_streams():
    """Step, chunk and mixed calls at once on their own streams give the bits
    that they give one after another."""
    import torch
    rng = np.random.default_rng(21)
    cache = make_cache(400, 2, 32, 128, "head", rng)
    tab = ints(rng.permutation(400).reshape(4, 100))
    lens = ints([3200, 1500, 33, 2999])
    qs = [torch.randn(n, 8, 128, device=DEV).bfloat16() for n in (4, 160, 4 + 70)]
    cus = [None, ints([0, 40, 80, 120, 160]), ints([0, 1, 2, 3, 74])]
    calls = [lambda s, q=q, c=c: fa.attention_forward_cache(q, cache, tab, lens, c, stream=s)
             for q, c in zip(qs, cus)]
    ref = []
    for c in calls:
        ref.append([t.clone() for t in c(None)])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    main = torch.cuda.current_stream()
    for s in streams:
        s.wait_stream(main)
    got = [(i % 3, calls[i % 3](s)) for _ in range(3) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, ref[i]))
    assert fa.fa_check(0) == fa.FA_OK


def test_calls_from_threads():
    """First and later calls from several host threads, each on its own stream."""
    import threading

    import torch
    rng = np.random.default_rng(22)
    cache = make_cache(60, 2, 16, 64, "head", rng)
    tab, lens = ints(np.arange(60).reshape(3, 20)), ints([300, 17, 120])
    q = torch.randn(3, 6, 64, device=DEV).half()
    ref = fa.attention_forward_cache(q, cache, tab, lens)
    torch.cuda.synchronize()
    out = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                r = fa.attention_forward_cache(q, cache, tab, lens, stream=s)
            s.synchronize()
        out[i] = r
    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert all(torch.equal(a, b) for r in out for a, b in zip(r, ref))


def test_outputs_and_queries_in_other_layouts():
    """q and o as views into wider rows (a fused projection), head-major and
    token-major."""
    import torch
    rng = np.random.default_rng(23)
    cache = make_cache(40, 2, 16, 128, "pair", rng)
    tab, lens = ints(np.arange(40).reshape(2, 20)), ints([310, 290])
    for n in (1, 6, 40):
        wide = torch.randn(2 * n, 3, 4, 128, device=DEV).bfloat16()
        q = wide[:, 1]
        cu = ints([0, n, 2 * n])
        ref = fa.attention_forward_cache(q.contiguous(), cache, tab, lens, cu)
        got = fa.attention_forward_cache(q, cache, tab, lens, cu)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        store = torch.zeros(2 * n, 4, 2, 128, device=DEV).bfloat16()
        o, lse = store[:, :, 0], torch.empty(2 * n, 4, device=DEV)
        ws = torch.empty(fa.fa_fwd_cache_workspace_size(2, 2 * n, 4, 2, 128), dtype=torch.uint8,
                         device=DEV)
        fa.attention_forward_cache_into(q, cache, tab, lens, o, lse, ws, cu)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
        assert (store[:, :, 1] == 0).all()


def test_binding_refusals():
    import torch
    c = fa.cache_empty(4, 2, 16, 64, device=DEV)
    i3 = ints([0, 1, 2])
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device=DEV)
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=DEV)
    tab, lens = ints(np.zeros((3, 2))), ints([1, 1, 1])
    with pytest.raises(ValueError):
        fa.cache_append(x, x, i3.long(), c)
    with pytest.raises(ValueError):
        fa.cache_append(x, x[:, :1], i3, c)
    with pytest.raises(ValueError):
        fa.cache_append(x, x.bfloat16(), i3, c)
    with pytest.raises(TypeError):
        fa.cache_append(x.float(), x.float(), i3, c)
    with pytest.raises(ValueError):
        fa.cache_append(x, x, i3, c._replace(v_scales=c.v_scales.double()))
    with pytest.raises(ValueError):
        fa.cache_append(x, x, i3, c._replace(k=c.k.cpu()))
    with pytest.raises(ValueError):
        fa.attention_forward_cache(q, c, tab, lens, ints([0, 1]))
    with pytest.raises(ValueError):
        fa.attention_forward_cache(q[:, :3], c, tab, lens)
    with pytest.raises(ValueError):
        fa.attention_forward_cache(q[:2], c, tab, lens)
    with pytest.raises(TypeError):
        fa.attention_forward_cache(q.float(), c, tab, lens)
    with pytest.raises(ValueError):
        fa.attention_forward_cache(q.transpose(1, 2), c, tab, lens)
    with pytest.raises(fa.FaError):
        fa.attention_forward_cache(q, c, tab, lens, scale=-1.0)
    with pytest.raises(fa.FaError):
        big = fa.cache_empty(2, 2, 24, 64, device=DEV)
        fa.cache_append(x, x, i3, big)
    # nothing to do is not an error
    fa.cache_append(x[:0], x[:0], i3[:0], c)
    o, lse = fa.attention_forward_cache(q[:0], c, tab, lens, ints([0, 0, 0, 0]))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_drafts_on_streams_and_at_a_largest_batch():
    """Drafts of 40 rows at once on several streams, bit for bit what they give alone;
    and 3000 sequences, of which every fifth has rows."""
    import torch
    rng = np.random.default_rng(21)
    H, heads, d, bs, B = 16, 2, 128, 32, 6
    lens = rng.integers(5, 900, B)
    need = -(-lens // bs)
    P = int(need.sum())
    cache = make_cache(P, heads, bs, d, "head", rng)
    table = np.full((B, int(need.max())), -1)
    ids, at = rng.permutation(P), 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    tab, ln, cu = ints(table), ints(lens), ints(np.arange(B + 1) * 5)
    qs = [torch.randn(5 * B, H, d, device=DEV).to(tdt(t)) for t in ("fp16", "bf16") * 3]
    alone = [fa.attention_forward_cache(q, cache, tab, ln, cu) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(3):
        got = [fa.attention_forward_cache(q, cache, tab, ln, cu, stream=st)
               for q, st in zip(qs, streams)]
        torch.cuda.synchronize()
        for (o, lse), (o1, l1) in zip(got, alone):
            assert torch.equal(o, o1) and torch.equal(lse, l1)
    counts = np.where(np.arange(3000) % 5 == 0, np.arange(3000) % 23, 0)
    lens = np.where(counts > 0, counts + np.arange(3000) % 40, np.arange(3000) % 2)
    attention_case(list(lens), list(counts), 2, 1, 32, 128, "bf16", True, seed=4)
