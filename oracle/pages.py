"""Plain sequential restatement of the page operators on numpy arrays: one row
after the other, one page at a time.  Each function returns (table, lens, refs,
pairs, info): the new books, the (source, destination) pages copied in order,
and the call's two info values; a call that fails returns the books as they
were, no pairs and its info.  Test infrastructure, never used by the library."""
from __future__ import annotations

import numpy as np


def _valid(table, lens, page, n_pages, refs=None):
    n, max_pages = table.shape
    for i in range(n):
        if not 0 <= lens[i] <= max_pages * page:
            return False
        for e in table[i, :-(-int(lens[i]) // page)]:
            if not 0 <= e < n_pages or (refs is not None and refs[e] <= 0):
                return False
    return True


def _refused(table, lens, refs, info):
    return table.copy(), lens.copy(), refs.copy(), [], info


def fork(table, lens, refs, parents, page):
    n, max_pages = table.shape
    if not _valid(table, lens, page, len(refs)) or any(not -1 <= p < n for p in parents):
        return _refused(table, lens, refs, (0, -1))
    new, new_lens, cnt = np.full_like(table, -1), np.zeros_like(lens), refs.copy()
    for i in range(n):  # every old row gives its pages back ...
        for e in table[i, :-(-int(lens[i]) // page)]:
            cnt[e] -= 1
    owed = []
    for i, p in enumerate(parents):  # ... and every new one takes what it shares
        if p < 0:
            continue
        new_lens[i] = lens[p]
        used = -(-int(lens[p]) // page)
        new[i, :used] = table[p, :used]
        keeper = p if parents[p] == p else list(parents).index(p)
        if lens[p] % page and keeper != i:
            owed.append((i, used - 1))
            used -= 1
        for e in new[i, :used]:
            cnt[e] += 1
    free = [p for p in range(len(refs)) if cnt[p] <= 0]
    if len(owed) > len(free):
        return _refused(table, lens, refs, (0, len(owed) - len(free)))
    pairs = []
    for (i, j), f in zip(owed, free):
        pairs.append((int(new[i, j]), f))
        new[i, j] = f
        cnt[f] = 1
    cnt[cnt < 0] = 0
    return new, new_lens, cnt, pairs, (len(owed), 0)


def resize(table, lens, refs, new_lens, page):
    n, max_pages = table.shape
    to = np.where(new_lens < 0, lens, new_lens)
    if not _valid(table, lens, page, len(refs)) or any(t > max_pages * page for t in to):
        return _refused(table, lens, refs, (0, -1))
    new, cnt = np.full_like(table, -1), refs.copy()
    for i in range(n):
        used, had = -(-int(to[i]) // page), -(-int(lens[i]) // page)
        new[i, :min(used, had)] = table[i, :min(used, had)]
        for e in table[i, used:had]:
            cnt[e] -= 1
    free = [p for p in range(len(refs)) if cnt[p] <= 0]
    pairs, at = [], 0
    for i in range(n):
        used, had = -(-int(to[i]) // page), -(-int(lens[i]) // page)
        places = list(range(had, used))
        if to[i] > lens[i] and lens[i] % page and cnt[table[i, had - 1]] > 1:
            cnt[table[i, had - 1]] -= 1
            places = [had - 1] + places
        for j in places:
            if at < len(free):
                if j < had:
                    pairs.append((int(table[i, j]), free[at]))
                new[i, j] = free[at]
                cnt[free[at]] = 1
            at += 1
    if at > len(free):
        return _refused(table, lens, refs, (0, at - len(free)))
    cnt[cnt < 0] = 0
    return new, to.astype(lens.dtype), cnt, pairs, (at, 0)


def compact(table, lens, refs, page):
    """As above, with the new id of every page before the info."""
    n_pages = len(refs)
    if not _valid(table, lens, page, n_pages, refs):
        moved = np.where(refs > 0, np.arange(n_pages), -1)
        return (*_refused(table, lens, refs, (0, -1))[:4], moved, (0, -1))
    live = [p for p in range(n_pages) if refs[p] > 0]
    moved, cnt, pairs = np.full(n_pages, -1), np.zeros_like(refs), []
    holes = iter([p for p in range(len(live)) if refs[p] <= 0])
    for p in live:
        moved[p] = p if p < len(live) else next(holes)
        cnt[moved[p]] = refs[p]
        if moved[p] != p:
            pairs.append((p, int(moved[p])))
    new = np.full_like(table, -1)
    for i in range(table.shape[0]):
        used = -(-int(lens[i]) // page)
        new[i, :used] = moved[table[i, :used]]
    return new, lens.copy(), cnt, pairs, moved, (len(live), len(pairs))


def copy_pairs(src_ids, dst_ids, n_src, n_dst, same):
    """The pairs that tq_pages_copy copies."""
    valid = [(int(s), int(t)) for s, t in zip(src_ids, dst_ids) if 0 <= s < n_src and 0 <= t < n_dst]
    sources = {s for s, _ in valid} if same else set()
    out, seen = [], set()
    for s, t in valid:
        if t not in seen and t not in sources:
            out.append((s, t))
        seen.add(t)
    return out
