"""Plain 64-bit references for the step operators: metadata from request
lengths, norm and rotation of queries and keys, the 4-bit cache and attention
over it.  numpy and loops only; nothing here calls the CUDA library."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.array([(8 + b % 8) / 8 * 2.0 ** (b // 8 - 7) if b > 7 else b / 8 * 2.0 ** -6 for b in range(127)])


# ------------------------------------------------------------------ metadata --

def step_metadata(ctx, new, tables, free, cursor, num_blocks, num_tokens):
    """Returns (tables, slots, positions, seq_lens, starts, cursor, bad) where
    bad is None, ("request", b) of some bad request, ("pages", needed) or
    ("step",)."""
    n, cols = tables.shape
    tables = tables.copy()
    bad, ok_ctx, ok_new = None, [], []
    for b, (c, q) in enumerate(zip(ctx, new)):
        c_ok = 0 <= c <= cols * 16
        valid = c_ok and q >= 0 and c + q <= cols * 16
        if not valid:
            bad = bad or ("request", b)
        ok_ctx.append(c if c_ok else 0)
        ok_new.append(q if valid else 0)
    need = [-(-(c + q) // 16) - -(-c // 16) for c, q in zip(ok_ctx, ok_new)]
    slots, positions = np.full(num_tokens, -1, np.int64), np.full(num_tokens, -1, np.int32)
    if not 0 <= cursor <= len(free) or sum(need) > len(free) - cursor or sum(ok_new) > num_tokens:
        if bad is None:
            bad = ("pages", sum(need)) if 0 <= cursor <= len(free) and sum(need) > len(free) - cursor else ("step",)
        return tables, slots, positions, np.array(ok_ctx, np.int32), np.zeros(n + 1, np.int32), cursor, bad
    starts, t = [0], 0
    for b in range(n):
        have = -(-ok_ctx[b] // 16)
        for j in range(need[b]):
            tables[b, have + j] = free[cursor]
            cursor += 1
        for i in range(ok_new[b]):
            pos = ok_ctx[b] + i
            page = int(tables[b, pos // 16])
            positions[t] = pos
            if 0 <= page < num_blocks:
                slots[t] = page * 16 + pos % 16
            else:
                bad = bad or ("request", b)
            t += 1
        starts.append(t)
    lens = np.array(ok_ctx, np.int32) + np.array(ok_new, np.int32)
    return tables, slots, positions, lens, np.array(starts, np.int32), cursor, bad


# -------------------------------------------------------- norm and rotation --

def norm_rope(x, weight, offset, eps, positions, cos_sin, interleaved):
    """x [T, H, Dh] float64 -> (result, bound on the 32-bit error's scale)."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (weight.astype(np.float64) + offset)
    y, size = x.copy(), np.abs(x)
    rot = cos_sin.shape[1]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    live = (positions >= 0) & (positions < len(cos_sin))
    row = cos_sin.astype(np.float64)[np.where(live, positions, 0)][:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


# --------------------------------------------------------------- 4-bit cache --

def _nearest_even(x, grid):
    """Index of the nearest grid value, a tie to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, x, side="left")
    tie = (i < len(mid)) & (mid[np.minimum(i, len(mid) - 1)] == x) & (i % 2 == 1)
    return i + tie


def quantise(x, tensor_scale):
    """x [..., Dh] -> codes [..., Dh] (0..15) and scale bytes [..., Dh/16]."""
    x = x.astype(np.float64) / tensor_scale
    blocks = x.reshape(x.shape[:-1] + (-1, 16))
    finite = np.isfinite(blocks).all(-1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = np.where(finite, np.abs(blocks).max(-1), 0.0)
        byte = np.where(finite, _nearest_even(top / 6, E4M3), 127).astype(np.uint8)
        s = np.where(finite, E4M3[np.minimum(byte, 126)], 1.0)[..., None]
        r = np.where(s > 0, np.abs(blocks) / s, 0.0)
    r = np.where(finite[..., None], r, 0.0)
    code = _nearest_even(r, E2M1).astype(np.uint8)
    code = np.where(finite[..., None], code + 8 * np.signbit(blocks), 0).astype(np.uint8)
    return code.reshape(x.shape), byte


def values(codes, scales, tensor_scale):
    """The values that codes [..., Dh] and scale bytes [..., Dh/16] stand for."""
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    v = np.concatenate([E2M1, -E2M1])[codes]
    return (v.reshape(v.shape[:-1] + (-1, 16)) * table[scales][..., None]).reshape(v.shape) * tensor_scale


def unpack(pool, which, dh):
    """Byte records [blocks, Hkv, 9*Dh] -> codes [blocks, 16, Hkv, Dh] and
    scales [blocks, 16, Hkv, Dh/16]."""
    n, h, _ = pool.shape
    body, sc = pool[..., :8 * dh], pool[..., 8 * dh:]
    if which == "k":
        body, sc = body.reshape(n, h, 16, dh // 2), sc.reshape(n, h, 16, dh // 16)
    else:
        body = body.reshape(n, h, dh // 2, 16).swapaxes(2, 3)
        sc = sc.reshape(n, h, dh // 16, 16).swapaxes(2, 3)
    codes = np.stack([body & 15, body >> 4], -1).reshape(n, h, 16, dh)
    return codes.swapaxes(1, 2), sc.swapaxes(1, 2)


def pool_values(pool, which, dh, tensor_scale):
    """[blocks, 16, Hkv, Dh] float64."""
    return values(*unpack(pool, which, dh), tensor_scale)


# ----------------------------------------------------------------- attention --

def attention(q, k_pages, v_pages, tables, lens, starts, scale):
    """out [T, Hq, Dh], lse [T, Hq], spread = sum_j p_j |v_j| [T, Hq, Dh] and
    reach = max_j scale * sum_d |q_d k_jd| [T, Hq], all float64, over pages
    [blocks, 16, Hkv, Dh].  Keys a query does not see take no part."""
    q = q.astype(np.float64)
    T, hq, dh = q.shape
    G = hq // k_pages.shape[2]
    out, spread = np.zeros((T, hq, dh)), np.zeros((T, hq, dh))
    lse, reach = np.zeros((T, hq)), np.zeros((T, hq))
    for b, n in enumerate(lens):
        s0, s1 = int(starts[b]), int(starts[b + 1])
        ids = [int(x) for x in tables[b][:-(-int(n) // 16)]]
        k = k_pages[ids].reshape(-1, *k_pages.shape[2:])[:n]
        v = v_pages[ids].reshape(-1, *v_pages.shape[2:])[:n]
        for i in range(s1 - s0):
            seen = int(n) - (s1 - s0) + i + 1
            for h in range(hq):
                kk, vv = k[:seen, h // G], v[:seen, h // G]
                z = kk @ q[s0 + i, h] * scale
                m = z.max()
                p = np.exp(z - m)
                out[s0 + i, h] = p @ vv / p.sum()
                spread[s0 + i, h] = p @ np.abs(vv) / p.sum()
                lse[s0 + i, h] = m + np.log(p.sum())
                reach[s0 + i, h] = (np.abs(kk) @ np.abs(q[s0 + i, h]) * scale).max()
    return out, lse, spread, reach
