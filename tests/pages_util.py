"""Plain implementations of the block cache's upkeep, one request after another on
the CPU, for the tests (numpy; no code of the library)."""
import numpy as np

from cache_util import CODE_VALUES, encode, pow2_above

LEAST = 2.0 ** -40


def counted(s):
    return pow2_above(float(s)) if s > 0 else 0.0


def keep(codes, scales, table, kv_lens, cu, words, bs):
    """(codes, scales, lens_out); codes [P, heads, bs, d], scales [P, heads], words: per
    sequence a list of 64-bit words."""
    codes, scales = codes.copy(), scales.astype(np.float64)
    P, heads = scales.shape
    out = []
    for b, length in enumerate(kv_lens):
        n = cu[b + 1] - cu[b]
        ok = 0 <= n <= length <= table.shape[1] * bs
        if ok and n:
            ids = table[b, (length - n) // bs: (length - 1) // bs + 1]
            ok = bool(((ids >= 0) & (ids < P)).all())
        if not ok:
            out.append(length)
            continue
        base = length - n
        path = [c for c in range(min(n, 64 * len(words[b]))) if words[b][c // 64] >> (c % 64) & 1]
        out.append(base + len(path))
        old_codes, old = codes.copy(), scales.copy()
        for j in range(base // bs, (base + len(path) - 1) // bs + 1 if path else 0):
            mine = [(k, c) for k, c in enumerate(path) if (base + k) // bs == j]
            if all(k == c for k, c in mine):
                continue
            page, older = table[b, j], max(base - j * bs, 0)
            for h in range(heads):
                from_ = [old[table[b, (base + c) // bs], h] for _, c in mine]
                now = max([counted(s) for s in from_] + ([counted(old[page, h])] if older else []))
                now = now if now > 0 else LEAST
                f = lambda s: s / now if s > 0 else 0.0  # noqa: E731
                for i in range(older):
                    codes[page, h, i] = bring(old_codes[page, h, i], f(old[page, h]))
                for (k, c), s in zip(mine, from_):
                    row = old_codes[table[b, (base + c) // bs], h, (base + c) % bs]
                    codes[page, h, (base + k) % bs] = bring(row, f(s))
                scales[page, h] = now
    return codes, scales, out


def bring(row, f):
    """Codes times f, as codes: the product is formed in 32 bits, which loses nothing where
    f is a power of two."""
    return row if f == 1.0 else encode((CODE_VALUES[row].astype(np.float32) * np.float32(f)).astype(np.float64))


def release(table, lens, new, free, pos, bs, shares=None):
    """(free, free_next, shares)."""
    free = list(free)
    shares = None if shares is None else list(shares)
    if not 0 <= pos <= len(free):
        return free, pos, shares
    entries = []
    for b in range(len(lens)):
        if 0 <= new[b] <= lens[b] <= table.shape[1] * bs:
            entries += [int(x) for x in table[b, -(-new[b] // bs): -(-lens[b] // bs)]]
    if shares is None:
        out = [x for x in entries if x >= 0]
    else:
        entries = [x for x in entries if 0 <= x < len(shares)]
        for x in entries:
            shares[x] -= 1
        out = []
        for x in entries:
            if shares[x] < 0 and x not in out:
                out.append(x)
        for x in out:
            shares[x] = 0
    for i, x in enumerate(out):
        if pos - 1 - i >= 0:
            free[pos - 1 - i] = x
    return free, max(pos - len(out), 0), shares


def fork(table, lens, src, free, pos, shares, bs):
    """(new_table, new_lens, copies, free_next, shares)."""
    width, shares = table.shape[1], list(shares)
    rows, out, copies, used, wanted = [], [], [], 0, 0
    for s in src:
        length = lens[s] if 0 <= s < len(lens) and 0 <= lens[s] <= width * bs else 0
        row = [-1] * width
        part = length % bs
        last = int(table[s, length // bs]) if part else -1
        needs = part > 0 and 0 <= last < len(shares)
        wanted += needs
        if needs and not (pos >= 0 and pos + wanted <= len(free)):
            length = 0
        copy = (-1, -1, 0)
        if length:
            for j in range(length // bs):
                row[j] = int(table[s, j])
                if 0 <= row[j] < len(shares):
                    shares[row[j]] += 1
            if needs:
                row[length // bs] = int(free[pos + used])
                copy = (last, row[length // bs], part)
                used += 1
            elif part:
                row[length // bs] = last
        rows.append(row)
        out.append(length)
        copies.append(copy)
    return np.array(rows), out, copies, pos + used, shares
