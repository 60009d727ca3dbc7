"""Plain sequential restatement of the step operators on numpy arrays: the slot
map of a step's tokens and the keeping of drafted rows.  Test infrastructure,
never used by the library."""
from __future__ import annotations

import numpy as np


def slots(table, lens, counts, page, n_pages, n_tokens, parents=None, words=0):
    """(cu_q, positions, slots, mask or None, status word)"""
    n = len(lens)
    cu = np.zeros(n + 1, np.int32)
    pos, slot = np.zeros(n_tokens, np.int32), np.full(n_tokens, -1, np.int64)
    mask = None if parents is None else np.zeros((n_tokens, words), np.uint32)
    for c, m in zip(counts, lens):
        if c < 0 or m < c or m > table.shape[1] * page or (parents is not None and c > 32 * words):
            return cu, pos, slot, mask, 63
    if int(np.sum(np.asarray(counts, np.int64))) > n_tokens:
        return cu, pos, slot, mask, 63
    status, t = 0, 0
    for b in range(n):
        first, base = t, int(lens[b]) - int(counts[b])
        sees = []
        for i in range(int(counts[b])):
            e = int(table[b, (base + i) // page])
            if 0 <= e < n_pages:
                slot[t] = e * page + (base + i) % page
            else:
                status = status or 64
            depth = i
            if parents is not None:
                p = int(parents[first + i])
                if not -1 <= p < i:
                    status, p = status or 65, -1
                sees.append((sees[p] if p >= 0 else 0) | 1 << i)
                depth = bin(sees[i]).count("1") - 1
                for w in range(words):
                    mask[t, w] = sees[i] >> 32 * w & 0xFFFFFFFF
            pos[t] = base + depth
            t += 1
        cu[b + 1] = t
    return cu, pos, slot, mask, status


def keep(table, lens, refs, counts, kept, n_keep, page, arrays):
    """(new lengths, the arrays after, status word); arrays: [n_pages, Hkv,
    page, ..] each, of any layer."""
    new, out, status = np.array(lens), [a.copy() for a in arrays], 0
    for b in range(len(lens)):
        n, k, base = int(counts[b]), int(n_keep[b]), int(lens[b]) - int(counts[b])
        ok = 0 <= n <= lens[b] <= table.shape[1] * page and 0 <= k <= min(n, kept.shape[1])
        moves = []
        for i in range(k if ok else 0):
            x = int(kept[b, i])
            if not i <= x < n or (i and x <= kept[b, i - 1]):
                ok = False
                break
            if x != i:
                a, z = int(table[b, (base + x) // page]), int(table[b, (base + i) // page])
                if not (0 <= a < len(refs) and 0 <= z < len(refs)) or refs[a] > 1 or refs[z] > 1:
                    ok = False
                    break
                moves.append((a, (base + x) % page, z, (base + i) % page))
        if not ok:
            status = 66
            continue
        new[b] = base + k
        for a, i, z, j in moves:  # ascending: no place is written before it is read
            for x in out:
                x[z, :, j] = x[a, :, i]
    return new, out, status
