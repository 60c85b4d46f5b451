"""Plain 64-bit implementations of the block cache's calls, on the CPU, for the
tests (numpy; no code of the library)."""
import math

import numpy as np

from attention_forward_flashattention_gb300 import inputs as I

MIN_EXP = -40
CODE_VALUES = I.e4m3_values()


def plan(lens, new, table, free, pos, T, bs):
    """(slots, cu, kv_lens, table, free_next) as lists / arrays: one request after another."""
    table = np.array(table, dtype=np.int64)
    slots = [-1] * T
    cu, kv, rows, wanted, used = [], [], 0, 0, 0
    for b, (x, m) in enumerate(zip(lens, new)):
        cu.append(min(rows, T))
        have, want = (max(x, 0) + bs - 1) // bs, (max(x, 0) + max(m, 0) + bs - 1) // bs
        ok = x >= 0 and m >= 0 and want <= table.shape[1] and x + m < 2 ** 31
        need = want - have if ok else 0
        wanted += need
        first = rows
        rows += max(m, 0)
        if m > 0 and rows > T:
            ok = False
        if need and not (0 <= pos and pos + wanted <= len(free)):
            ok = False
        if ok:
            for j in range(need):
                table[b, have + j] = free[pos + used + j]
            used += need
            for i in range(m):
                at = x + i
                page = int(table[b, at // bs])
                slot = page * bs + at % bs
                slots[first + i] = slot if page >= 0 and slot < 2 ** 31 else -1
        kv.append(x + m if ok else max(x, 0))
    cu.append(min(rows, T))
    return slots, cu, kv, table, pos + used


def need_scale(amax):
    if amax <= 0:
        return 2.0 ** MIN_EXP
    e = max(math.ceil(math.log2(amax / 448.0)) - 1, MIN_EXP)   # at or one below the wanted one
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def pow2_above(x):
    m, e = math.frexp(x)
    return 2.0 ** (e - 1 if m == 0.5 else e)


def encode(x):
    """e4m3 codes of float64 values; infinities and NaN give NaN."""
    bad = ~np.isfinite(x)
    codes = I.to_e4m3_bits(np.where(bad, 0.0, x))
    return np.where(bad, np.uint8(0x7F), codes)


def append(x, slots, codes, scales, bs):
    """Appends x [T, heads, d] (float64 values) to codes [P, heads, bs, d] and
    scales [P, heads]; returns new ones."""
    codes, scales = codes.copy(), scales.astype(np.float64)
    P, heads = scales.shape
    T = len(slots)
    t = 0
    while t < T:
        s = int(slots[t])
        if not 0 <= s < P * bs:
            t += 1
            continue
        n = 1
        while t + n < T and slots[t + n] == s + n and (s + n) % bs:
            n += 1
        p, off = divmod(s, bs)
        for h in range(heads):
            v = x[t:t + n, h]
            fine = np.abs(v[np.isfinite(v)])
            now = need_scale(fine.max() if fine.size else 0.0)
            if off:
                old = scales[p, h]
                now = max(now, pow2_above(old))
                if now != old:
                    codes[p, h, :off] = encode(CODE_VALUES[codes[p, h, :off]] * (old / now))
            scales[p, h] = now
            codes[p, h, off:off + n] = encode(v / now)
        t += n
    return codes, scales


def attend(q, k, v, ks, vs, table, kv_lens, cu, bs, scale, causal):
    """float64 attention. q [T, H, d] values, k, v codes [P, Hkv, bs, d]. Returns
    (O, LSE, mag, far, small): mag = the weighted mean of |v|, far = the
    largest bound on a score's fp32 error over the row's keys (natural units),
    small = 2^-25 sum |v code| times the largest V scale (the weights' fp16
    subnormals)."""
    T, H, d = q.shape
    P, heads = ks.shape
    g = H // heads
    O = np.zeros((T, H, d))
    L = np.full((T, H), -np.inf)
    mag, far, small = np.zeros((T, H, d)), np.zeros((T, H)), np.zeros((T, H))
    width = table.shape[1] * bs
    for b, length in enumerate(kv_lens):
        length = min(max(int(length), 0), width)
        r0, r1 = cu[b], cu[b + 1]
        n = r1 - r0
        ids = np.array([table[b, j // bs] for j in range(length)], dtype=np.int64)
        seen = (ids >= 0) & (ids < P)
        safe = np.where(seen, ids, 0)
        at = np.arange(length) % bs
        for h in range(heads):
            kk = CODE_VALUES[k[safe, h, at]].reshape(length, d) * ks[safe, h][:, None]
            vc = CODE_VALUES[v[safe, h, at]].reshape(length, d)
            vv = vc * vs[safe, h][:, None]
            for i in range(n):
                lim = min(length, length - n + i + 1) if causal else length
                keep = np.flatnonzero(seen[:max(lim, 0)])
                if keep.size == 0:
                    continue
                for j in range(g):
                    row, head = r0 + i, h * g + j
                    s = kk[keep] @ q[row, head] * scale
                    top = s.max()
                    p = np.exp(s - top)
                    O[row, head] = p @ vv[keep] / p.sum()
                    L[row, head] = top + math.log(p.sum())
                    mag[row, head] = p @ np.abs(vv[keep]) / p.sum()
                    far[row, head] = ((d + 3) * 2.0 ** -24 * scale
                                      * (np.abs(kk[keep]) @ np.abs(q[row, head])).max())
                    small[row, head] = (2.0 ** -25 * np.abs(vc[keep]).sum(axis=0).max()
                                        * vs[safe, h][keep].max())
    return O, L, mag, far, small


def attend_tolerance(ref, eps, keys):
    """Bounds on |O - ref| and |LSE - ref|. Weights: rounded to fp16 (half a
    step, 2^-11), a score's fp32 error `far` twice (numerator and sum), the
    exponential and the fp32 sums over the keys (keys * 2^-24 and 2^-20); O is
    rounded to its type once (eps / 2). LSE: the score, the sum, and fp32
    values of up to |LSE| + 64 in size."""
    O, L, mag, far, small = ref
    rel = 2.0 ** -11 + 2 * far + keys * 2.0 ** -24 + 2.0 ** -20
    tol_o = mag * rel[..., None] * (1 + eps) + np.abs(O) * (eps / 2) + small[..., None] + 1e-30
    # results below the type's normal range have a fixed step
    tol_o = tol_o + (2.0 ** -25 if eps == 2.0 ** -10 else 0.0)
    lf = np.where(np.isfinite(L), np.abs(L), 0.0)
    tol_l = far + keys * 2.0 ** -24 + 2.0 ** -20 + 8 * 2.0 ** -24 * (lf + 64)
    return tol_o, tol_l


def attend_columns(q, k, v, ks, vs, table, kv_lens, cu, bs, scale, causal, eps, two_parts=False,
                   q_floor=0.0):
    """float64 attention with bounds on the error of every single result, from the
    terms that it is made of. Arguments as in attend; eps: of the results' type;
    two_parts: weights kept as two fp16 values; q_floor: rounding of a query
    element, relative to the largest one of its row. Returns (O, LSE, tol_O, tol_LSE).

    With w_j = exp(s_j), W = max w_j vs_j and L = sum w_j:
    - a weight's relative error r_j: the score's fp32 sum, (d + 3) 2^-24 scale
      sum |k q| and q_floor's share; the fp32 exponent c s + log2 vs - m, 2^-23 of
      the magnitudes that it is formed of, and 2^-22 of log2 vs; 2^-20 for the
      exponential and the scales' reciprocal. It enters numerator and L.
    - its rounding for the product with V: 2^-11 of itself (two parts: 2^-22), or
      2^-33 W where that is more (both kernels' references lie 2^-8 or more below the
      largest weight, and fp16's half step below its normal range is 2^-25).
    - the fp32 sums over the keys: 2^-24 for each of them in numerator and L, 2^-14
      at most (a share of the keys is summed by itself, by MMAs of 16 keys).
    - O is rounded to its type once; fp16 has a fixed step of 2^-24 below 2^-14."""
    T, H, d = q.shape
    P, heads = ks.shape
    g = H // heads
    O, tol_o = np.zeros((T, H, d)), np.full((T, H, d), 1e-300)
    L, tol_l = np.full((T, H), -np.inf), np.zeros((T, H))
    width = table.shape[1] * bs
    part = 2.0 ** -22 if two_parts else 2.0 ** -11
    for b, length in enumerate(kv_lens):
        length = min(max(int(length), 0), width)
        n = cu[b + 1] - cu[b]
        at = np.arange(length)
        ids = table[b, at // bs] if length else np.zeros(0, dtype=np.int64)
        seen = (ids >= 0) & (ids < P)
        safe = np.where(seen, ids, 0)
        for h in range(heads):
            kk = CODE_VALUES[k[safe, h, at % bs]] * ks[safe, h][:, None]
            vc = CODE_VALUES[v[safe, h, at % bs]]
            sv = vs[safe, h]
            for i in range(n):
                lim = min(length, length - n + i + 1) if causal else length
                keep = np.flatnonzero(seen[:max(lim, 0)])
                if keep.size == 0:
                    continue
                kj, vj, sj = kk[keep], vc[keep], sv[keep]
                lv = np.log2(sj)
                sums = min(keep.size * 2.0 ** -24, 2.0 ** -14)
                for j in range(g):
                    t, head = cu[b] + i, h * g + j
                    x = q[t, head]
                    s = kj @ x * scale
                    e = s * math.log2(math.e) + lv
                    r = ((d + 3) * 2.0 ** -24 * scale * (np.abs(kj) @ np.abs(x))
                         + q_floor * scale * np.abs(x).max() * np.abs(kj).sum(-1)
                         + math.log(2) * (2.0 ** -23 * (np.abs(e) + np.abs(lv) + np.abs(e.max()) + 11)
                                          + 2.0 ** -22 * np.abs(lv))
                         + 2.0 ** -20)
                    w = np.exp(s - s.max())
                    tot = w.sum()
                    u = w * sj                       # what a code is multiplied by
                    O[t, head] = u @ vj / tot
                    L[t, head] = s.max() + math.log(tot)
                    rl = (w * np.expm1(r)).sum() / tot + sums
                    du = np.maximum(u * part, 2.0 ** -33 * u.max()) + u * (np.expm1(r) + sums)
                    tol_o[t, head] += (du @ np.abs(vj) / tot + np.abs(O[t, head]) * rl) * (1 + eps)
                    tol_o[t, head] += np.abs(O[t, head]) * eps / 2
                    # LSE = ln 2 (m + log2 l): fp32, and log2's own error
                    tol_l[t, head] = rl + 2.0 ** -22 * (np.abs(L[t, head]) + np.abs(e.max()) + 64)
    if eps == 2.0 ** -10:
        tol_o += 2.0 ** -25
    return O, L, tol_o, tol_l
