"""Page tables and slot maps of a paged key cache, one step (oracle; test infrastructure only).

The definition, request by request and token by token: finished requests push their pages on the
stack of free pages, then every request pops the pages its new tokens need, and each new token's
cache row is its page times the page size plus its offset.  A step that cannot be done whole
changes nothing and maps nothing.

Pinned by: a hand-worked step, and the invariants (no page held twice, pages conserved).
"""

import numpy as np

ST_NO_PAGES, ST_BAD_LEN = 16, 32


def page_step(lens, new, done, table, free_list, count, page_size, max_new):
    """Returns a dict of the arrays after the step; the inputs are left alone."""
    n, max_pages = table.shape
    out = dict(table=table.copy(), free_list=free_list.copy(), lens=lens.copy(), count=int(count),
               row_begin=np.zeros(n + 1, np.int32), slot=np.full(max_new, -1, np.int64),
               row=np.full(max_new, -1, np.int32), pos=np.full(max_new, -1, np.int32), status=0)
    pages = lambda tokens: -(-int(tokens) // page_size)
    kept = [0 if done[r] else int(lens[r]) for r in range(n)]
    room = max_pages * page_size
    bad = any(lens[r] < 0 or new[r] < 0 or lens[r] > room or kept[r] + int(new[r]) > room
              for r in range(n))
    total = 0 if bad else sum(int(x) for x in new)
    if bad or total > max_new:
        out["status"] |= ST_BAD_LEN
    if not bad:
        back = sum(pages(lens[r]) for r in range(n) if done[r])
        need = sum(pages(kept[r] + int(new[r])) - pages(kept[r]) for r in range(n))
        if count < 0 or count + back > len(free_list) or need > count + back:
            out["status"] |= ST_NO_PAGES
    if out["status"]:
        return out
    top = int(count)
    for r in range(n):
        if done[r]:
            for i in range(pages(lens[r])):
                out["free_list"][top] = table[r, i]
                top += 1
    t = 0
    for r in range(n):
        out["row_begin"][r] = t
        end = kept[r] + int(new[r])
        for i in range(pages(kept[r]), pages(end)):
            top -= 1
            out["table"][r, i] = out["free_list"][top]
        for p in range(kept[r], end):
            out["slot"][t] = int(out["table"][r, p // page_size]) * page_size + p % page_size
            out["row"][t], out["pos"][t] = r, p
            t += 1
        out["lens"][r] = end
    out["row_begin"][n] = t
    out["count"] = top
    return out
