"""A bad page id in pa_paged_attention_scored reaches the rows that see a key of the
page and no others: not those of other requests whose work shares its CTAs."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_scored_attention import _batch, _slopes

pytestmark = pytest.mark.gpu

RULES = {"plain": {}, "cap": dict(soft_cap=20.0), "bias": dict(slopes=True)}


def _run(a, rules):
    rules = {k: _slopes(a["q"].shape[1]) if v is True else v for k, v in rules.items()}
    out, lse = pa.paged_attention_scored(**a, **rules)
    return out, lse, pa.check_errors()


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 256), (4, 1, 512)])
@pytest.mark.parametrize("rule", list(RULES))
def test_a_bad_page_changes_nothing_for_who_does_not_see_it(rule, heads):
    """Many requests share CTAs with one whose table has a bad id: their rows, and its
    rows that do not see the page, have the bits that they have with a sound table."""
    lens = [300] * 150 + [1000]
    new = [90] * 150 + [1000]
    a = _batch(lens, new, *heads, seed=3)
    rules = dict(RULES[rule], window=50)
    clean = _run(a, rules)
    assert clean[2] == (0, -1)
    a["block_tables"][70, 17] = 10**6        # keys 272 .. 287
    a["block_tables"][150, 40] = -1          # keys 640 .. 655
    bad = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    starts = a["query_start_loc"].tolist()
    for b, k0 in ((70, 272), (150, 640)):
        pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
        bad[starts[b]:starts[b + 1]] = (pos >= k0) & (pos - 50 < k0 + 15)
    for _ in range(4):
        out, lse, st = _run(a, rules)
        assert st[0] == pa.PA_ERR_BAD_METADATA and st[1] in (70, 150)
        assert torch.equal(out.isnan().flatten(1).all(1), bad) and torch.equal(lse.isnan().all(1), bad)
        assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 256), (4, 1, 512)])
def test_every_id_of_a_long_request_is_bad(heads):
    """All of its rows are NaN, and quickly so; the other requests keep their bits."""
    lens, new = [200] * 20 + [30000] + [200] * 20, [200] * 20 + [700] + [200] * 20
    a = _batch(lens, new, *heads, seed=5)
    clean = _run(a, {})
    a["block_tables"][20] = 2**31 - 1
    out, lse, st = _run(a, {})
    assert st == (pa.PA_ERR_BAD_METADATA, 20)
    rows = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    rows[20 * 200:20 * 200 + 700] = True
    assert out[rows].isnan().all() and lse[rows].isnan().all()
    assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse[~rows], clean[1][~rows])
