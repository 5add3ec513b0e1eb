"""Tokens that see nothing between tokens that see keys, in one tile of rows: pages
that no token of the request sees may hold anything, and so may their table entries."""
import math

import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_scored_attention import POISON, _batch, _check, i32

pytestmark = pytest.mark.gpu

BAD = [POISON, -1, -7, 10**7]


def _gap(lens, new, lo, hi, heads, seed, nan_pages):
    """Of each request's tokens those at positions n - new + lo .. n - new + hi - 1 see
    nothing, and the ones behind them nothing before position n - new + hi."""
    a = _batch(lens, [new] * len(lens), *heads, seed=seed)
    first = []
    for b, n in enumerate(lens):
        base = n - new
        first += [0] * lo + [base + i + 1 for i in range(lo, hi)] + [base + hi] * (new - hi)
        for page in range(-(-(base + lo) // 16), (base + hi) // 16):
            if nan_pages:
                at = int(a["block_tables"][b, page])
                a["k_cache"][at], a["v_cache"][at] = math.nan, math.nan
            else:
                a["block_tables"][b, page] = BAD[page % 4]
    return a, dict(first_keys=i32(first))


@pytest.mark.parametrize("heads,new", [((8, 2, 128), 64), ((8, 2, 128), 300), ((4, 4, 128), 32), ((1, 1, 128), 32),
                                       ((3, 1, 256), 40), ((4, 1, 256), 64), ((1, 1, 512), 32), ((2, 1, 512), 64)])
@pytest.mark.parametrize("nan_pages", [False, True])
def test_gaps_inside_a_tile(heads, new, nan_pages):
    for lens in ([new, 512 + new], [700, 333, 16 + new]):
        lo, hi = 3, new - 5
        a, rules = _gap(lens, new, lo, hi, heads, 1, nan_pages)
        _check(a, rules)
        _check(a, dict(soft_cap=30.0, **rules))


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 512)])
def test_two_gaps_and_a_prefix(heads):
    """A prefix that reaches into the first gap, a window, and a second gap."""
    n, new = 256, 120
    a = _batch([n], [new], *heads, seed=2)
    base = n - new
    first = [0] * 4 + [POISON] * 40 + [base + 44] * 8 + [POISON] * 60 + [base + 112] * 8
    prefix = base + 20
    seen = set(range(prefix)) | {base + i for i in (*range(4), *range(44, 52), *range(112, 120))}
    pages = [p for p in range(n // 16) if not seen & set(range(16 * p, 16 * p + 16))]
    assert len(pages) >= 3
    for i, p in enumerate(pages):
        a["block_tables"][0, p] = BAD[i % 4]
    _check(a, dict(first_keys=i32(first), prefix_lens=i32([prefix])))
    _check(a, dict(first_keys=i32(first), prefix_lens=i32([prefix]), window=30, soft_cap=20.0))


# (in the first the gap is keys 515 .. 570, in the second 671 .. 694: pages 33, 34 and 42)
@pytest.mark.parametrize("heads,n,new,sound,token", [((8, 2, 128), 576, 64, 10, 17), ((1, 1, 128), 700, 32, 2, 5)])
def test_a_bad_page_that_one_token_of_a_gap_sees_is_named(heads, n, new, sound, token):
    a, rules = _gap([n], new, 3, new - 5, heads, 3, False)
    base = n - new
    rules["first_keys"][sound] = base + sound          # sees itself alone, in a sound page
    out, lse = pa.paged_attention_scored(**a, **rules)
    assert pa.check_errors() == (0, -1) and bool(out[sound].isfinite().all())
    assert (base + token) // 16 in (33, 42)
    rules["first_keys"][token] = base + token          # in a page whose entry is bad
    out, lse = pa.paged_attention_scored(**a, **rules)
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 0)
    bad = torch.zeros(new, dtype=torch.bool)
    bad[token] = True
    assert torch.equal(out.isnan().flatten(1).all(1).cpu(), bad) and torch.equal(out.isnan().flatten(1).any(1).cpu(), bad)
    assert torch.equal(lse.isnan().all(1).cpu(), bad)
