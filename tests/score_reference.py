"""A plain 64-bit reference of attention with rules for the scores, request by
request and head by head; nothing here calls the CUDA library.  Runs on the
tensors' device."""
from __future__ import annotations

import math

import torch


def seen_keys(n, new, window=0, prefix=0, first=None, device="cpu"):
    """[new, n] bool: which keys the last `new` of n tokens see."""
    j = torch.arange(n, device=device)
    p = torch.arange(n - new, n, device=device).unsqueeze(1)
    see = j <= p
    if window:
        see &= p - j < window
    if first is not None:
        see &= j >= first.to(device).long().unsqueeze(1)
    return see | (j < prefix)


def attention(q, k_cache, v_cache, tables, lens, starts, scale, soft_cap=0.0, slopes=None, window=0, prefix_lens=None,
              first_keys=None, small_cap_error=False):
    """out [T, Hq, Dh], lse [T, Hq] and the bounds of a 32-bit computation's
    error, all float64.  Hidden keys take no part, whatever they hold.

    The bounds.  A score is a sum of Dh products accumulated in 32 bits, each
    step off by at most 2^-23 of the largest partial sum (reach = scale * sum
    |q_d k_d|); the cap adds 2^-21 of itself, scaling, bias and exponent 2^-22 of
    the largest magnitude among them: together `delta`, an error of the exponent.
    Probabilities are rounded to BF16 (2^-8 of each), the result too:
      out: 2^-8 |out| + (2^-8 + 2 delta) sum_j p_j |v_j|, twice delta for the sum;
      lse: delta + n 2^-24 (a chain of n additions) + 2^-22 |lse|.
    With small_cap_error a cap above 56 adds 2^-19 of the capped score instead:
    0.358 of the cap and more (|z| > 3/8 of it) are good to 2.3 units of 2^-22 of the
    cap, less to a dozen roundings of themselves."""
    T, hq, dh = q.shape
    group = hq // k_cache.shape[2]
    dev = q.device
    out = torch.zeros((T, hq, dh), dtype=torch.float64, device=dev)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=dev)
    tol_out, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(int(x) for x in lens):
        s0, s1 = int(starts[b]), int(starts[b + 1])
        if s1 == s0:
            continue
        pages = tables[b, :-(-n // 16)].long()
        see = seen_keys(n, s1 - s0, window, 0 if prefix_lens is None else min(max(int(prefix_lens[b]), 0), n),
                        None if first_keys is None else first_keys[s0:s1], dev)
        used = see.any(0)
        # pages without a seen key may be anything: take page 0 for them and hide it
        live = torch.nn.functional.pad(used, (0, pages.numel() * 16 - n)).view(-1, 16).any(1)
        pages = torch.where(live, pages, torch.zeros_like(pages))
        k = k_cache[pages].flatten(0, 1)[:n].double()
        v = v_cache[pages].flatten(0, 1)[:n].double()
        k[~used], v[~used] = 0, 0
        j = torch.arange(n, device=dev)
        p = torch.arange(n - (s1 - s0), n, device=dev).unsqueeze(1)
        dist = (p - j).abs().double()
        near = torch.where(see, dist, torch.full_like(dist, 1e18)).min(1, keepdim=True).values
        for h in range(hq):
            kk, vv, x = k[:, h // group], v[:, h // group], q[s0:s1, h].double()
            z = x @ kk.T * scale
            reach = x.abs() @ kk.abs().T * scale
            if soft_cap:
                z = soft_cap * torch.tanh(z / soft_cap)
            size = z_cap = z.abs()
            if slopes is not None:
                bias = slopes[h].double() * dist
                size = torch.maximum(size, (bias - slopes[h].double() * near).abs())
                z = z - bias
            of_cap = soft_cap * 2.0**-21 if soft_cap <= 56 or not small_cap_error else z_cap * 2.0**-19
            delta = reach * dh * 2.0**-23 + of_cap + size * 2.0**-22 + 2.0**-21
            z = torch.where(see, z, torch.full_like(z, -math.inf))
            lse[s0:s1, h] = torch.logsumexp(z, 1)
            w = torch.where(see, torch.exp(z - lse[s0:s1, h, None]), torch.zeros_like(z))
            finite = torch.isfinite(vv).all(1)
            vv = torch.where(finite[:, None], vv, torch.zeros_like(vv))  # (0 times it would be NaN for who does not see it)
            out[s0:s1, h] = w @ vv
            out[s0:s1, h][(see & ~finite).any(1)] = math.nan
            top = (w > 2.0**-40) & see  # (what weighs nothing adds no error worth the name)
            d = torch.where(top, delta, torch.zeros_like(delta)).max(1).values
            tol_out[s0:s1, h] = 2.0**-8 * out[s0:s1, h].abs() + (2.0**-8 + 2 * d[:, None]) * (w @ vv.abs()) + 1e-30
            tol_lse[s0:s1, h] = d + see.sum(1) * 2.0**-24 + 2.0**-22 * lse[s0:s1, h].abs().nan_to_num(posinf=0)
    return out, lse, tol_out, tol_lse
