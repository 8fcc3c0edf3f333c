"""Plain Python oracle of the paged cache's page operators -- TEST INFRASTRUCTURE.

Each function works on copies, one row, pair or page at a time, and returns the
new state and the status bits.  It shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

BAD_INDEX, OVERFLOW, BAD_LENGTH = 1, 4, 8


def _free(refs):
    return [p for p in range(len(refs)) if refs[p] == 0]


def oracle_resize_pages(table, held, refs, new_lens, page_size):
    """Rows shrink, then grow by the lowest free pages in row order.  Returns
    (table, held, refs, status)."""
    table, held, refs = table.copy(), held.copy(), refs.copy()
    N, width, status = len(refs), table.shape[1], 0
    want = {}
    for r in range(len(held)):
        w = int(held[r]) if new_lens[r] < 0 else -(-int(new_lens[r]) // page_size)
        if held[r] < 0 or held[r] > width or w > width:
            status |= BAD_LENGTH
        else:
            want[r] = w
    for r, w in want.items():
        for j in range(w, int(held[r])):
            p = int(table[r, j])
            table[r, j] = -1
            if p < 0 or p >= N or refs[p] <= 0:
                status |= BAD_INDEX
            else:
                refs[p] -= 1
        held[r] = min(held[r], w)
    free, full = _free(refs), False
    for r, w in want.items():
        k = w - int(held[r])
        if k <= 0:
            continue
        if full or k > len(free):
            full = True
            status |= OVERFLOW
            continue
        for j in range(k):
            table[r, held[r] + j] = free[j]
            refs[free[j]] = 1
        free = free[k:]
        held[r] = w
    return table, held, refs, status


def oracle_fork_pages(k_pool, v_pool, table, held, refs, ctx, parent, child):
    """Pools [layers, pages, page_size, ...].  Returns (k_pool, v_pool, table, held,
    refs, ctx, status)."""
    old_held, old_ctx, old_table, old_refs = held.copy(), ctx.copy(), table.copy(), refs.copy()
    k_pool, v_pool = k_pool.copy(), v_pool.copy()
    table, held, refs, ctx = table.copy(), held.copy(), refs.copy(), ctx.copy()
    R, page, N, status = len(held), k_pool.shape[2], len(refs), 0
    free, taken, shared = _free(refs), set(), []
    for p, c in zip(parent.tolist(), child.tolist()):
        if p < 0:
            continue
        if p >= R or not 0 <= c < R or p == c or c in taken or old_held[c] != 0:
            status |= BAD_INDEX
            if 0 <= c < R:
                taken.add(c)
            continue
        taken.add(c)
        n = int(old_ctx[p])
        if n < 0 or old_held[p] > table.shape[1] or -(-n // page) > old_held[p]:
            status |= BAD_LENGTH
            continue
        full, part = n // page, n % page
        if part:
            if not free:
                status |= OVERFLOW
                continue
            new, last = free.pop(0), int(old_table[p, full])
            table[c, full] = new
            refs[new] = 1
            if 0 <= last < N and old_refs[last] != 0:
                k_pool[:, new, :part] = k_pool[:, last, :part]
                v_pool[:, new, :part] = v_pool[:, last, :part]
            else:
                status |= BAD_INDEX
        for j in range(full):
            q = int(old_table[p, j])
            table[c, j] = q
            if 0 <= q < N and old_refs[q] != 0:
                shared.append(q)
            else:
                status |= BAD_INDEX
        held[c], ctx[c] = full + (part > 0), n
    for q in shared:
        refs[q] += 1
    return k_pool, v_pool, table, held, refs, ctx, status


def oracle_copy_pages(k_pool, v_pool, src, dst):
    """Pools [layers, pages, ...].  Returns (k_pool, v_pool, status)."""
    N, status = k_pool.shape[1], 0
    real = []
    for i, (s, d) in enumerate(zip(src.tolist(), dst.tolist())):
        if s < 0 or (s == d and s < N):
            continue
        if s >= N or not 0 <= d < N:
            status |= BAD_INDEX
        else:
            real.append((i, s, d))
    k_new, v_new = k_pool.copy(), v_pool.copy()
    for i, s, d in real:
        if any((t == d and k < i) or t == s for k, _, t in real):
            status |= BAD_INDEX
            continue
        k_new[:, d], v_new[:, d] = k_pool[:, s], v_pool[:, s]
    return k_new, v_new, status


def oracle_compact_pages(k_pool, v_pool, table, held, refs):
    """Returns (k_pool, v_pool, table, refs, remap, n_live, status)."""
    N, status = len(refs), 0
    n_live = int(np.count_nonzero(refs))
    holes = [p for p in range(n_live) if refs[p] == 0]
    moving = [p for p in range(n_live, N) if refs[p] != 0]
    remap = np.where(refs != 0, np.arange(N), -1).astype(np.int32)
    k_new, v_new, table, refs = k_pool.copy(), v_pool.copy(), table.copy(), refs.copy()
    for d, s in zip(holes, moving):
        k_new[:, d], v_new[:, d] = k_pool[:, s], v_pool[:, s]
        refs[d], refs[s] = refs[s], 0
        remap[s] = d
    for r in range(len(held)):
        for j in range(min(int(held[r]), table.shape[1])):
            p = int(table[r, j])
            if 0 <= p < N and remap[p] >= 0:
                table[r, j] = remap[p]
            else:
                status |= BAD_INDEX
    return k_new, v_new, table, refs, remap, n_live, status
