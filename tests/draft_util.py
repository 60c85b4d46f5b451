"""Plain 64-bit trees of drafted tokens and their attention over a block cache, on
the CPU, for the tests (numpy; no code of the library)."""
import math

import numpy as np

from cache_util import CODE_VALUES


def masks_of(parents, cu, lens, words):
    """(masks [T, words] as Python ints of each word, positions [T]); rows of no request are None."""
    T = len(parents)
    masks, positions = [None] * T, [None] * T
    for b in range(len(lens)):
        lo, hi = (min(max(cu[b + x], 0), T) for x in (0, 1))
        sets = []
        for i in range(max(hi - lo, 0)):
            p = parents[lo + i]
            # (a token without a bit has no ancestors either)
            sets.append(((sets[p] if 0 <= p < i else set()) | {i}) if i < 64 * words else set())
            masks[lo + i] = [sum(1 << c % 64 for c in sets[i] if c // 64 == w) for w in range(words)]
            positions[lo + i] = max(lens[b], 0) + max(len(sets[i]) - 1, 0)
    return masks, positions


def signed(words):
    """64-bit words as int64 values."""
    a = np.array(words, dtype=object)
    return np.where(a >= 2 ** 63, a - 2 ** 64, a).astype(np.int64)


def seen(masks, length, n, i):
    """The keys that query i of n sees, as truth values [length]; masks: its words."""
    out = np.ones(length, dtype=bool)
    for key in range(max(length - n, 0), length):
        c = key - (length - n)
        out[key] = c < 64 * len(masks) and bool(masks[c // 64] >> (c % 64) & 1)
    return out


def attend(q, k, v, ks, vs, table, kv_lens, cu, masks, bs, scale, eps, two_parts=False, q_floor=0.0):
    """(O, LSE, tol_O, tol_LSE): attention with masks, and bounds on the error of every
    result from the terms that it is made of, the same as for the causal attention
    (cache_util.attend_columns tells them): r_j for each weight's relative error,
    its rounding to 11 (two parts: 22) bits or 2^-33 of the row's largest, fp32 sums,
    one rounding of O."""
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
        there = (ids >= 0) & (ids < P)
        safe = np.where(there, ids, 0)
        for h in range(heads):
            kk = CODE_VALUES[k[safe, h, at % bs]] * ks[safe, h][:, None]
            vc = CODE_VALUES[v[safe, h, at % bs]]
            sv = vs[safe, h]
            for i in range(n):
                t = cu[b] + i
                keep = np.flatnonzero(there & seen(masks[t], length, n, i))
                if keep.size == 0:
                    continue
                kj, vj, sj = kk[keep], vc[keep], sv[keep]
                lv = np.log2(sj)
                sums = min(keep.size * 2.0 ** -24, 2.0 ** -14)
                x = q[t, h * g:(h + 1) * g]                       # [g, d]
                s = x @ kj.T * scale                              # [g, keys]
                e = s * math.log2(math.e) + lv
                top = e.max(1, keepdims=True)
                r = ((d + 3) * 2.0 ** -24 * scale * (np.abs(x) @ np.abs(kj).T)
                     + q_floor * scale * np.abs(x).max(1, keepdims=True) * np.abs(kj).sum(-1)
                     + math.log(2) * (2.0 ** -23 * (np.abs(e) + np.abs(lv) + np.abs(top) + 11)
                                      + 2.0 ** -22 * np.abs(lv)) + 2.0 ** -20)
                w = np.exp(s - s.max(1, keepdims=True))
                tot = w.sum(1, keepdims=True)
                u = w * sj
                o = u @ vj / tot
                lse = s.max(1) + np.log(tot[:, 0])
                rl = (w * np.expm1(r)).sum(1, keepdims=True) / tot + sums
                du = np.maximum(u * part, 2.0 ** -33 * u.max(1, keepdims=True)) + u * (np.expm1(r) + sums)
                rows = slice(h * g, (h + 1) * g)
                O[t, rows], L[t, rows] = o, lse
                tol_o[t, rows] += (du @ np.abs(vj) / tot + np.abs(o) * rl) * (1 + eps) + np.abs(o) * eps / 2
                tol_l[t, rows] = rl[:, 0] + 2.0 ** -22 * (np.abs(lse) + np.abs(top[:, 0]) + 64)
    if eps == 2.0 ** -10:
        tol_o += 2.0 ** -25
    return O, L, tol_o, tol_l
