"""Attention over latent rows in float64, the blocks that scores select, the weight each token got and
its accumulation into the pool's eviction order (oracle; test infrastructure only).

A latent row is 576 values, a token's key for every head; its first 512 are the token's value.  Every
function walks tokens one list at a time, straight from the definition.

Readings: a token listed twice counts twice; positions at or behind a row's length, behind the page
table or the cache are no tokens; a row without a token gives zeros and a log sum of -infinity.

Pinned by: hand-worked softmaxes of one, two and equal tokens, invariance under the order of the list,
joining of two halves by their log sums, and weights that add up to the number of heads.
"""

import numpy as np

VALUES = 512


def listed_rows(idx, block, n_kv, length=None, table=None, page_size=0, req=None):
    """For each row of idx: (places in the list, rows of the cache) of its tokens."""
    out = []
    for r, entries in enumerate(np.asarray(idx)):
        places, rows = [], []
        for i, e in enumerate(entries):
            if e < 0:
                continue
            for b in range(block):
                p = int(e) * block + b
                if length is not None and p >= length[r]:
                    continue
                if table is not None:
                    t = r if req is None else int(req[r])
                    if not 0 <= t < len(table) or p // page_size >= table.shape[1]:
                        continue
                    page = int(table[t, p // page_size])
                    if page < 0:
                        continue
                    p = page * page_size + p % page_size
                if 0 <= p < n_kv:
                    places.append(i * block + b)
                    rows.append(p)
        out.append((np.array(places, np.int64), np.array(rows, np.int64)))
    return out


def paged_rows(length, pages, page_size, n_kv):
    """Cache rows of the first `length` positions of one page list."""
    p = np.arange(max(0, int(length)))
    p = p[p // page_size < len(pages)]
    pg = np.asarray(pages, np.int64)[p // page_size]
    at = pg * page_size + p % page_size
    return at[(pg >= 0) & (at < n_kv)]


def prefix_rows(n_rows, n_kv, page_size, group_begin, prefix_len, prefix_table, own_len, own_table):
    """Cache rows that each row of the batch attends to: its group's prefix, then its own."""
    out = []
    for r in range(n_rows):
        rows = [paged_rows(own_len[r], own_table[r], page_size, n_kv)]
        for g in range(len(prefix_len)):
            if group_begin[g] <= r < group_begin[g + 1]:
                rows.insert(0, paged_rows(prefix_len[g], prefix_table[g], page_size, n_kv))
        out.append(np.concatenate(rows))
    return out


def attention(q, kv, rows, scale):
    """q [R, H, 576], kv [n, 576] float64, rows: a list of cache rows for each query row.
    (out, lse, weighted sizes of the values [R, H, 512], largest sum of |products| behind a score [R, H])"""
    R, H = q.shape[:2]
    out, lse = np.zeros((R, H, VALUES)), np.full((R, H), -np.inf)
    size, terms = np.zeros((R, H, VALUES)), np.zeros((R, H))
    for r in range(R):
        k = kv[rows[r]]
        if not len(k):
            continue
        s = scale * (q[r] @ k.T)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(1, keepdims=True)
        lse[r] = (m + np.log(z))[:, 0]
        out[r] = (p / z) @ k[:, :VALUES]
        size[r] = (p / z) @ np.abs(k[:, :VALUES])
        terms[r] = abs(scale) * (np.abs(q[r]) @ np.abs(k).T).max(1)
    return out, lse, size, terms


def token_weights(q, kv, places, rows, lse, scale, n):
    """What each of a row's n list places got from all heads."""
    w = np.zeros((len(rows), n))
    for r in range(len(rows)):
        s = scale * (q[r] @ kv[rows[r]].T)
        w[r, places[r]] = np.exp(s - lse[r][:, None]).sum(0)
    return w


def block_topk(scores, length, block, k, n_first=0, n_last=0):
    """idx [rows, k]: the k blocks of the largest token scores, ties to the lower block, ascending, -1 padded."""
    out = np.full((len(length), k), -1, np.int32)
    for r, n in enumerate(length):
        n = max(0, min(int(n), scores.shape[1]))
        nb = -(-n // block)
        m = np.array([scores[r, b * block:min(n, (b + 1) * block)].max() for b in range(nb)], np.float64)
        m[:n_first] = np.inf
        m[max(0, nb - n_last):] = np.inf
        take = np.sort(np.lexsort((np.arange(nb), -m))[:k])
        out[r, :len(take)] = take
    return out


def weigh(mass, free, slot, w, decay, fresh=()):
    """(mass, priority) after a step: float32 arithmetic as documented, sums in units of 2^-32."""
    f = np.float32
    n = len(mass)
    units = np.zeros(n, object)
    for s, x in zip(np.ravel(slot), np.ravel(w)):
        if 0 <= s < n:
            x = 0.0 if np.isnan(x) else min(max(float(x), 0.0), 1024.0)
            units[s] += int(np.rint(x * 2.0 ** 32))
    old = np.where(mass > 0, mass, f(0)).astype(f) * f(decay)
    for s in np.ravel(fresh):
        if 0 <= s < n:
            old[s] = 0
    # a whole number of up to 63 bits to the nearest float32, then the scale, which is exact
    add = np.array([_to_f32(int(u)) for u in units], f) * f(2.0 ** -32)
    new = (old + add).astype(f)
    new[np.asarray(free) != 0] = 0
    priority = np.where(np.asarray(free) != 0, -1, new.view(np.int32)).astype(np.int32)
    return new, priority


def _to_f32(u):
    """The float32 nearest to a whole number, ties to even (through a double it would be rounded twice)."""
    bits = u.bit_length()
    if bits <= 24:
        return float(u)
    sh = bits - 24
    q, rest = u >> sh, u & ((1 << sh) - 1)
    half = 1 << (sh - 1)
    if rest > half or (rest == half and q & 1):
        q += 1
    return float(q) * 2.0 ** sh
