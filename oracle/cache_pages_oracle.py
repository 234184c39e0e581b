"""Plain models of the cache's page operators, one step at a time in the order that the header
gives them. Caches are byte arrays [L, pages, page bytes]; tables are Python-sized numpy arrays
changed in place. Every function returns the error bits it would set."""
from __future__ import annotations

import numpy as np

ERR_INDEX, ERR_PAGE = 1, 2
ROW = {"bf16": 1152, "fp8_ds": 656, "fp8_tensor": 576, "index_keys": 128}


def page_bytes(fmt: str, P: int) -> int:
    return P * (132 if fmt == "index_keys" else ROW[fmt])


def row_get(cache, fmt, P, page, k):
    """Bytes of row k of a page in every layer (index keys: codes and scale)."""
    R = ROW[fmt]
    a = cache[:, page, k * R:(k + 1) * R]
    if fmt == "index_keys":
        a = np.concatenate([a, cache[:, page, 128 * P + 4 * k:128 * P + 4 * k + 4]], axis=1)
    return a.copy()


def row_set(cache, fmt, P, page, k, v):
    R = ROW[fmt]
    cache[:, page, k * R:(k + 1) * R] = v[:, :R]
    if fmt == "index_keys":
        cache[:, page, 128 * P + 4 * k:128 * P + 4 * k + 4] = v[:, R:]


def copy_pages(cache, src, dst):
    err, n = 0, cache.shape[1]
    old = cache.copy()
    for s, d in zip(src, dst):
        if s == -1 or d == -1 or s == d:
            continue
        if not (0 <= s < n and 0 <= d < n):
            err |= ERR_PAGE
            continue
        cache[:, d] = old[:, s]
    return err


def compact(cache, fmt, P, table, starts, cu, keep, lens=None):
    err, num_pages, stride = 0, cache.shape[1], table.shape[1]
    for r in range(len(starts)):
        a, b, st = int(cu[r]), int(cu[r + 1]), int(starts[r])
        if st < 0 or a < 0 or b < a or b > len(keep) or st + b - a > 2**31 - 1:
            err |= ERR_INDEX
            continue
        for k in range(b - a):
            src = int(keep[a + k])
            prev = int(keep[a + k - 1]) if k else -1
            if src < k or src <= prev:
                err |= ERR_INDEX
                continue
            if src == k:
                continue
            place = []
            for slot in (st + src, st + k):
                if slot // P >= stride:
                    err |= ERR_INDEX
                    continue
                page = int(table[r, slot // P])
                if not 0 <= page < num_pages:
                    err |= ERR_PAGE
                    continue
                place.append((page, slot % P))
            if len(place) == 2:
                row_set(cache, fmt, P, *place[1], row_get(cache, fmt, P, *place[0]))
        if lens is not None:
            lens[r] = st + b - a
    return err


def fork(cache, fmt, P, table, lens, refs, free, count, src, dst):
    """Returns (error bits, new free count, fork_pages)."""
    err, B, stride, num_pages = 0, len(lens), table.shape[1], len(refs)
    pages, asked = [], 0
    for i, (s, d) in enumerate(zip(src, dst)):
        s, d = int(s), int(d)
        ok = 0 <= s < B and 0 <= d < B
        ok = ok and list(dst).count(d) == 1 and d not in list(src) and lens[d] == 0 and 0 <= lens[s] <= stride * P
        if not ok:
            err |= ERR_INDEX
            pages.append(-2)
            continue
        n = int(lens[s])
        got = -1
        if n % P:
            if not 0 <= int(table[s, n // P]) < num_pages:  # nothing to copy the rows from
                err |= ERR_PAGE
                pages.append(-2)
                continue
            asked += 1
            if asked > count:
                err |= ERR_PAGE
                pages.append(-2)
                continue
            got = int(free[count - asked])
            free[count - asked] = -1
            if not 0 <= got < num_pages:
                err |= ERR_PAGE
                pages.append(-2)
                continue
            refs[got] = 1
            table[d, n // P] = got
            old = int(table[s, n // P])
            for k in range(n % P):
                row_set(cache, fmt, P, got, k, row_get(cache, fmt, P, old, k))
        for k in range(n // P):
            page = int(table[s, k])
            table[d, k] = page
            if 0 <= page < num_pages:
                refs[page] += 1
            else:
                err |= ERR_PAGE
        lens[d] = n
        pages.append(got)
    return err, count - min(asked, count), pages


def resize(P, table, lens, refs, free, count, req, new):
    """Returns (error bits, new free count)."""
    err, B, stride, num_pages = 0, len(lens), table.shape[1], len(refs)
    good, freed = [], []
    for r, m in zip(req, new):
        ok = 0 <= r < B and list(req).count(r) == 1 and 0 <= m <= stride * P and 0 <= lens[r] <= stride * P
        good.append(ok)
        if not ok:
            err |= ERR_INDEX
            continue
        for k in range(-(-int(m) // P), -(-int(lens[r]) // P)):
            page = int(table[r, k])
            table[r, k] = -1
            if not 0 <= page < num_pages or refs[page] <= 0:
                err |= ERR_PAGE
                continue
            refs[page] -= 1
            if refs[page] == 0:
                freed.append(page)
    for page in sorted(freed):
        free[count] = page
        count += 1
    avail, asked, given = count, 0, 0
    for ok, r, m in zip(good, req, new):
        if not ok:
            continue
        a, b = -(-int(lens[r]) // P), -(-int(m) // P)
        need = max(0, b - a)
        asked += need
        if need and asked > avail:
            err |= ERR_PAGE
            continue
        for k in range(a, b):
            page = int(free[count - 1])
            free[count - 1] = -1
            count -= 1
            if not 0 <= page < num_pages:  # no page: the slots stay without one
                err |= ERR_PAGE
                page = -1
            else:
                refs[page] = 1
            table[r, k] = page
        lens[r] = m
    return err, count
