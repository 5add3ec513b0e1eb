"""Caps far above the scores, as large as the call takes: a capped score is good to
a few roundings of itself, not of the cap."""
import math

import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import score_reference as ref
from tests.test_gpu_scored_attention import _batch, _slopes, i32

pytestmark = pytest.mark.gpu

CAPS = [30.0, 55.0, 57.0, 400.0, 2.0**16, 2.0**18, 2.0**20]
SHAPES = {
    "decode": ([1, 17, 700, 2049], [1, 1, 1, 1]),
    "drafts": ([18, 260, 1030], [2, 4, 3]),
    "chunks": ([33, 515, 900], [20, 257, 64]),
}


def _check(a, rules, keep=slice(None)):
    out, lse = pa.paged_attention_scored(**a, **rules)
    assert pa.check_errors() == (0, -1)
    want, want_lse, tol, tol_lse = ref.attention(a["q"], a["k_cache"], a["v_cache"], a["block_tables"],
                                                 a["seq_lens"].tolist(), a["query_start_loc"].tolist(), a["scale"],
                                                 small_cap_error=True, **rules)
    worst = ((out.double() - want).abs() / tol)[..., keep].max().item()
    assert worst <= 1, ("out", worst)
    worst = ((lse.double() - want_lse).abs() / tol_lse).max().item()
    assert worst <= 1, ("lse", worst)


@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 2, 256), (4, 1, 512)])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("cap", CAPS)
def test_scores_far_below_the_cap(cap, shape, heads):
    a = _batch(*SHAPES[shape], *heads, seed=1)
    _check(a, dict(soft_cap=cap))
    _check(a, dict(soft_cap=cap, slopes=_slopes(heads[0]), window=300))


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("cap", CAPS)
def test_scores_around_the_cap(cap, shape):
    """Spread so that scores lie on both sides of 3/8 of the cap."""
    a = _batch(*SHAPES[shape], 8, 2, 128, seed=2, spread=0.5 * min(cap, 400.0))
    _check(a, dict(soft_cap=cap))
    _check(a, dict(soft_cap=cap, slopes=_slopes(8)))


@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("cap", [57.0, 2.0**20])
def test_rows_computed_key_by_key(cap, new):
    """One infinite value that all rows see: its column is infinite, the others and
    lse are as good as without it."""
    a = _batch([400], [new], 8, 2, 128, seed=3)
    page = int(a["block_tables"][0, 1])
    a["v_cache"][page, 5, :, 7] = 0
    clean = {k: v.clone() if k == "v_cache" else v for k, v in a.items()}
    a["v_cache"][page, 5, :, 7] = math.inf
    rules = dict(soft_cap=cap)
    out, lse = pa.paged_attention_scored(**a, **rules)
    assert bool((out[..., 7] == math.inf).all())
    want, want_lse, tol, tol_lse = ref.attention(clean["q"], clean["k_cache"], clean["v_cache"], a["block_tables"], [400],
                                                 [0, new], a["scale"], small_cap_error=True, **rules)
    others = [d for d in range(128) if d != 7]
    assert bool(((out.double() - want).abs() <= tol)[..., others].all())
    assert bool(((lse.double() - want_lse).abs() <= tol_lse).all())


def test_the_prefix_alone():
    a = _batch([2000], [3], 8, 2, 128, seed=4)
    _check(a, dict(soft_cap=2.0**20, first_keys=i32([2000] * 3), prefix_lens=i32([90]), slopes=_slopes(8)))
