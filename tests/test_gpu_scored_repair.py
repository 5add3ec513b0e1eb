"""Rows whose result is not finite beside rows whose is, in pa_paged_attention_scored:
the same bits every time, and nothing changes for who does not see the cause."""
import math

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


# one group to many CTAs, many groups to a CTA, both; one row tile and two
BATCHES = [([1500], [40]), ([1500], [600]), ([90] * 200, [90] * 200), ([700, 300, 1200], [700, 20, 33])]


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 256), (16, 1, 256), (4, 1, 512)])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("rule", list(RULES))
def test_one_bad_column_and_the_same_bits_every_time(rule, batch, heads):
    """An infinity in one column of a value: every repeat gives the same bits, lse is
    what it is without it (it does not depend on values), and rows that do not see
    the key keep their results within the rounding of the probabilities."""
    lens, new = BATCHES[batch]
    a = _batch(lens, new, *heads, seed=1)
    rules = dict(RULES[rule], window=64)
    clean = _run(a, rules)
    for b, n in enumerate(lens):
        j = n - new[b] // 2 - 1
        a["v_cache"][int(a["block_tables"][b, j // 16]), j % 16, :, (7 * b + 40) % heads[2]] = math.inf
    first = _run(a, rules)
    assert first[2] == (0, -1) and torch.equal(first[1], clean[1])
    for _ in range(8):
        again = _run(a, rules)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])
    starts = a["query_start_loc"].tolist()
    for b, n in enumerate(lens):
        j, d = n - new[b] // 2 - 1, (7 * b + 40) % heads[2]
        pos = torch.arange(n - new[b], n, device="cuda")
        sees = (pos >= j) & (pos - j < 64)
        rows = slice(starts[b], starts[b + 1])
        got, want = first[0][rows], clean[0][rows]
        assert bool((got[sees][..., d] == math.inf).all()), b
        finite = got.isfinite()
        finite[..., d] |= sees[:, None]
        assert bool(finite.all()), b
        # (both are within 2^-8 of the value and 2^-8 of the values' size, here below 4)
        err = torch.where(got.isfinite(), (got.double() - want.double()).abs(), torch.zeros((), dtype=torch.float64, device="cuda"))
        assert bool((err <= 2.0**-6 * (want.double().abs() + 4)).all()), b


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 512)])
def test_columns_of_other_owners_keep_their_bits(heads):
    """Head dim 512: the halves of the columns are computed apart; a part of a group:
    32 columns at a time.  Who owns sound columns stores what it stores without the
    bad one."""
    a = _batch([1500], [40 if heads[2] == 128 else 100], *heads, seed=2)
    clean = _run(a, {})
    a["v_cache"][int(a["block_tables"][0, 3]), 1, :, 1] = math.inf
    out, lse, _ = _run(a, {})
    assert bool((out[..., 1] == math.inf).all()) and torch.equal(lse, clean[1])
    from_ = 32 if heads[2] == 128 else 256
    assert torch.equal(out[..., from_:], clean[0][..., from_:])


def test_rows_that_take_seconds_latch_nothing():
    """Two groups of 256 rows over 262144 keys to a CTA; an infinity that all rows of
    the first see: they are computed again key by key, which takes longer than any
    wait between warps may last."""
    n, new, hq, dh, count = 262144, 32, 8, 128, 304
    pages = n // 16
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.randn(pages + 1, 2, 16, 1, dh, generator=g, device="cuda").to(torch.bfloat16)
    pool[pages] = pool[0]
    pool[pages, 1, 5, 0, 9] = math.inf
    tables = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(count, 1)
    tables[::2, 0] = pages
    q = torch.randn(new, hq, dh, generator=g, device="cuda").to(torch.bfloat16).repeat(count, 1, 1)
    a = dict(q=q, k_cache=pool[:, 0], v_cache=pool[:, 1], block_tables=tables,
             seq_lens=torch.full((count,), n, dtype=torch.int32, device="cuda"),
             query_start_loc=torch.arange(0, count * new + 1, new, dtype=torch.int32, device="cuda"), scale=dh**-0.5,
             max_query_len=new, max_seq_len=n)
    out, lse, st = _run(a, {})
    assert st == (0, -1)
    out, lse = out.unflatten(0, (count, new)), lse.unflatten(0, (count, new))
    assert bool((out[::2, ..., 9] == math.inf).all()) and bool(out[1::2].isfinite().all())
    assert torch.equal(lse, lse[:1].expand_as(lse))
    clean = out[1].double()
    for b in range(count):
        if b % 2:
            assert torch.equal(out[b], out[1])
            continue
        # (both are within 2^-8 of the value and of sum p |v|, which is below 1)
        err = (out[b].double() - clean).abs()
        err[..., 9] = 0
        assert bool((err <= 2.0**-6).all())


SHAPES = {"few": ([700, 33, 1, 260], [1, 1, 1, 1], 8, 2, 128), "many": ([300, 513, 40], [300, 200, 40], 8, 2, 128),
          "wide": ([600, 70], [600, 3], 4, 1, 512), "one_tile": ([400] * 40, [9] * 40, 6, 1, 256)}


@pytest.mark.parametrize("pinned", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_a_captured_call_with_and_without_the_cause(shape, pinned):
    """Replays see an infinity, a bad page, nothing, in turn: each gives what a call by
    itself gives, and nothing of the one before stays."""
    lens, new, *heads = SHAPES[shape]
    a = _batch(lens, new, *heads, seed=4)
    T, hq, dh = a["q"].shape
    out, lse = torch.empty(T, hq, dh, dtype=torch.bfloat16), torch.empty(T, hq)
    out, lse = (t.pin_memory() if pinned else t.cuda() for t in (out, lse))
    ws = pa.new_scored_workspace(len(lens), hq, heads[1], dh, a["max_query_len"], a["max_seq_len"])
    pa.init()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call = pa.prepare_paged_attention_scored(**a, out=out, lse=lse, workspace=ws, soft_cap=20.0, window=100, stream=st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    j = lens[0] - new[0] // 2 - 1
    value, entry = a["v_cache"][int(a["block_tables"][0, j // 16]), j % 16], a["block_tables"][0, j // 16]
    sound, page = value.clone(), entry.clone()
    for cause in ("none", "value", "page", "none", "page", "value"):
        value.copy_(sound)
        entry.copy_(page)
        if cause == "value":
            value[..., 3] = math.inf
        if cause == "page":
            entry.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        status = pa.check_errors()
        want = pa.paged_attention_scored(**a, soft_cap=20.0, window=100)
        assert status == pa.check_errors() == ((pa.PA_ERR_BAD_METADATA, 0) if cause == "page" else (0, -1))
        assert torch.equal(out.cuda().view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(lse.cuda().view(torch.int32), want[1].view(torch.int32))
        assert bool(want[0].isfinite().all()) == (cause == "none")


@pytest.mark.parametrize("shape", list(SHAPES))
def test_without_lse(shape):
    lens, new, *heads = SHAPES[shape]
    a = _batch(lens, new, *heads, seed=5)
    j = lens[0] - new[0] // 2 - 1
    a["v_cache"][int(a["block_tables"][0, j // 16]), j % 16, :, 3] = math.inf
    want, _ = pa.paged_attention_scored(**a)
    out, lse = pa.paged_attention_scored(**a, want_lse=False)
    assert lse is None and torch.equal(out, want) and not bool(out.isfinite().all())


CAUSES = {"up": (math.inf,), "down": (-math.inf,), "nan": (math.nan,), "both": (math.inf, -math.inf), "up_nan": (math.inf, math.nan)}


@pytest.mark.parametrize("cause", list(CAUSES))
@pytest.mark.parametrize("shape", list(SHAPES))
def test_who_sees_values_that_are_not_finite(shape, cause):
    """They have them in that column, who sees none of them has a number there; other
    columns are as good as without them, and lse keeps its bits."""
    lens, new, *heads = SHAPES[shape]
    a = _batch(lens, new, *heads, seed=6)
    out, lse = pa.paged_attention_scored(**a, window=60)
    clean = out.clone(), lse.clone()
    base = lens[0] - new[0]
    keys = [max(base - 20, 0), max(base - 20, 0) + 7][:len(CAUSES[cause])]
    for j, value in zip(keys, CAUSES[cause]):
        a["v_cache"][int(a["block_tables"][0, j // 16]), j % 16, :, 17] = value
    got = pa.paged_attention_scored(**a, window=60)
    assert pa.check_errors() == (0, -1)
    others = [d for d in range(heads[2]) if d != 17]
    assert torch.equal(got[1], clean[1])
    # (both are within 2^-8 of the value and 2^-8 of the values' size, here below 4)
    x, y = got[0][..., others].double(), clean[0][..., others].double()
    assert bool(((x - y).abs() <= 2.0**-6 * (y.abs() + 4)).all())
    column, was = got[0][..., 17], clean[0][..., 17]
    for t in range(out.shape[0]):
        pos = base + t
        seen = [v for j, v in zip(keys, CAUSES[cause]) if t < new[0] and j <= pos and pos - j < 60]
        if not seen:
            assert bool(((column[t].double() - was[t].double()).abs() <= 2.0**-6 * (was[t].double().abs() + 4)).all()), t
        elif len(set(seen)) == 1 and not math.isnan(seen[0]):
            assert bool((column[t] == seen[0]).all()), t
        else:
            assert bool(column[t].isnan().all()), t


@pytest.mark.parametrize("key,slope", [(35, 1.0), (299, -1.0)])
@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 1, 256), (2, 1, 512)])
def test_an_infinity_of_little_weight(heads, new, key, slope):
    """A weight below the smallest of 32 bits (of keys behind it, or before it, that
    weigh more) is not zero: the column is infinite."""
    a = _batch([400], [new], *heads, seed=7)
    a["v_cache"][int(a["block_tables"][0, key // 16]), key % 16, :, 70] = -math.inf
    out, lse = pa.paged_attention_scored(**a, slopes=torch.full((heads[0],), slope, device="cuda"))
    assert pa.check_errors() == (0, -1) and bool(lse.isfinite().all())
    assert bool((out[..., 70] == -math.inf).all()) and bool(out[..., :70].isfinite().all())


def test_a_sum_that_overflows_before_its_division():
    """Values near the largest: the sum of weight times value passes 32 bits, the
    result does not."""
    for heads, new in (((8, 2, 128), 300), ((4, 1, 256), 300), ((4, 1, 512), 40), ((8, 2, 128), 1)):
        a = _batch([600], [new], *heads, seed=8)
        for page in a["block_tables"][0, :38].tolist():
            v = a["v_cache"][page]
            v[..., 5] = torch.where(v[..., 5].isnan(), v[..., 5], torch.full_like(v[..., 5], 3e38))
        out, lse = pa.paged_attention_scored(**a)
        assert pa.check_errors() == (0, -1) and bool(out.isfinite().all())
        # (2^-8 of the result, 2^-8 of the sum's probabilities, all of one sign)
        assert bool(((out[..., 5].double() / 3e38 - 1).abs() <= 2.0**-6).all())
