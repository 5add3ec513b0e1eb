"""Plain references of the calls that move pages between requests: loops over
requests and columns, numpy only; nothing here calls the CUDA library."""
from __future__ import annotations

import numpy as np


def pages(n):
    return -(-int(n) // 16)


def fork(parents, children, lens, ctx, tables, shares, free, cursor, num_blocks):
    """Returns (tables, shares, seq_lens, cursor, src, dst, bad); bad is None,
    ("fork", i), ("pages", needed) or ("call",)."""
    tables, shares, out = tables.copy(), shares.copy(), np.array(ctx, np.int32)
    n, cols = len(parents), tables.shape[1]
    src, dst = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    bad, good, taken = None, [], set()
    for i, (p, c) in enumerate(zip(parents, children)):
        ok = 0 <= p < len(ctx) and 0 <= c < len(ctx) and c not in taken and ctx[c] == 0
        if 0 <= c < len(ctx):
            taken.add(c)
        ok = ok and 0 <= ctx[p] <= cols * 16
        n_tok = None if not ok else ctx[p] if lens is None else lens[i]
        ok = ok and 0 <= n_tok <= ctx[p]
        if ok:
            good.append((i, int(p), int(c), int(n_tok)))
        else:
            bad = bad or ("fork", i)
    need = sum(1 for g in good if g[3] % 16)
    if not 0 <= cursor <= len(free) or need > len(free) - cursor:
        if bad is None:
            bad = ("pages", need) if 0 <= cursor <= len(free) else ("call",)
        return tables, shares, out, cursor, src, dst, bad
    for i, p, c, n_tok in good:
        out[c] = n_tok
        for j in range(n_tok // 16):
            tables[c, j] = tables[p, j]
            if 0 <= tables[p, j] < num_blocks:
                shares[tables[p, j]] += 1
            else:
                bad = bad or ("fork", i)
        if n_tok % 16:
            new, old = int(free[cursor]), int(tables[p, n_tok // 16])
            cursor += 1
            tables[c, n_tok // 16] = new
            if 0 <= new < num_blocks and 0 <= old < num_blocks:
                src[i], dst[i] = old, new
            else:
                bad = bad or ("fork", i)
    return tables, shares, out, cursor, src, dst, bad


def release(ctx, keep, tables, shares, free, cursor, num_blocks):
    """Returns (shares, free, seq_lens, cursor, bad); bad is None, ("request", b),
    ("pages", freed) or ("call",)."""
    start, shares, free = shares, shares.copy(), free.copy()
    out, bad, gone, freed = np.array(ctx, np.int32), None, [], {}  # (freed: in order)
    for b, (c, k) in enumerate(zip(ctx, keep)):
        ok = 0 <= c <= tables.shape[1] * 16 and k <= c
        if ok and 0 <= k < c:
            if k % 16:
                p = tables[b, k // 16]
                ok = 0 <= p < num_blocks and start[p] == 0
            if ok:
                out[b] = k
                gone += [(b, int(p)) for p in tables[b, pages(k):pages(c)]]
        if not ok:
            bad = bad or ("request", b)
    for b, p in gone:
        if not 0 <= p < num_blocks:
            bad = bad or ("request", b)
            continue
        shares[p] -= 1
        if shares[p] < 0:
            if p in freed:
                bad = bad or ("request", b)
            else:
                freed[p] = True
    if not 0 <= cursor <= len(free) or len(freed) > cursor:
        if bad is None:
            bad = ("pages", len(freed)) if 0 <= cursor <= len(free) else ("call",)
        return start.copy(), free, np.array(ctx, np.int32), cursor, bad
    freed = list(freed)
    shares[freed] = 0
    cursor -= len(freed)
    free[cursor:cursor + len(freed)] = freed
    return shares, free, out, cursor, bad


def compact(ctx, tables, shares, free, cursor, num_blocks, max_moves):
    """Returns (tables, shares, free, cursor, src, dst, counts, bad)."""
    tables, free = tables.copy(), free.copy()
    bad, used = None, set()
    rows = []
    for b, c in enumerate(ctx):
        if not 0 <= c <= tables.shape[1] * 16:
            bad = bad or ("request", b)
            continue
        rows.append((b, pages(c)))
        for p in tables[b, :pages(c)]:
            if 0 <= p < num_blocks:
                used.add(int(p))
            else:
                bad = bad or ("request", b)
    n = len(used)
    movers = sorted(p for p in used if p >= n)
    holes = sorted(set(range(n)) - used)
    src, dst = np.full(max_moves, -1, np.int32), np.full(max_moves, -1, np.int32)
    counts = np.array([n, len(movers)], np.int32)
    if len(movers) > max_moves:
        return tables, shares.copy(), free, cursor, src, dst, counts, bad or ("moves", len(movers))
    src[:len(movers)], dst[:len(movers)] = movers, holes
    place = dict(zip(movers, holes))
    for b, m in rows:
        tables[b, :m] = [place.get(int(p), int(p)) for p in tables[b, :m]]
    out = np.zeros_like(shares)
    for p in used:
        out[place.get(p, p)] = shares[p]
    shift = len(free) - num_blocks
    free[shift + n:] = np.arange(n, num_blocks)
    return tables, out, free, shift + n, src, dst, counts, bad
