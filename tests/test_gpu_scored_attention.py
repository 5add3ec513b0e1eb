"""pa_paged_attention_scored on the GPU against the 64-bit reference: rules by
themselves and together, head layouts, lengths at the edges of pages and tiles,
rows that see nothing, garbage in everything that is not seen, errors."""
import math

import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import score_reference as ref

pytestmark = pytest.mark.gpu

POISON = 2**31 - 1
i32 = lambda x: torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _batch(lens, new, hq, hkv, dh, seed=0, layout="interleaved", spread=1.0):
    """A pool that holds NaN but for the requests' tokens, shuffled tables with
    garbage past the last page, padded query rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = [-(-n // 16) for n in lens]
    nb = sum(pages) + 5
    if layout == "interleaved":
        pool = torch.full((nb, 2, 16, hkv, dh), math.nan, dtype=torch.bfloat16, device="cuda")
        k, v = pool[:, 0], pool[:, 1]
    else:  # head-major, apart
        k, v = (torch.full((nb, hkv, 16, dh), math.nan, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
                for _ in range(2))
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    cols = max(pages + [1]) + 2
    tables = torch.full((len(lens), cols), POISON, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        ids = perm[at:at + pages[b]]
        tables[b, :pages[b]] = ids
        at += pages[b]
        for c in (k, v):
            x = torch.randn(pages[b] * 16, hkv, dh, generator=g, device="cuda").to(torch.bfloat16)
            x[n:] = math.nan
            c[ids.long()] = x.view(pages[b], 16, hkv, dh)
    T = sum(new)
    qbuf = torch.randn(max(T, 1), hq * dh + 8, generator=g, device="cuda").mul_(spread).to(torch.bfloat16)
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    return dict(q=qbuf[:T, :hq * dh].unflatten(1, (hq, dh)), k_cache=k, v_cache=v, block_tables=tables, seq_lens=i32(lens),
                query_start_loc=i32(starts), scale=1 / math.sqrt(dh), max_query_len=max(new), max_seq_len=max(lens))


def _slopes(hq):
    return 2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float32, device="cuda") / hq)


def _rules(name, lens, new, hq):
    T = sum(new)
    pos = [n - x + i for n, x in zip(lens, new) for i in range(x)]
    some = {
        "plain": {},
        "cap": dict(soft_cap=20.0),
        "bias": dict(slopes=_slopes(hq)),
        "window": dict(window=37),
        "window1": dict(window=1),
        "sinks": dict(window=100, prefix_lens=i32([4] * len(lens))),
        "prefix": dict(prefix_lens=i32([min(n, 13 + 50 * b) for b, n in enumerate(lens)])),
        "docs": dict(first_keys=i32([p - p % (31 + 70 * (p % 3 > 0)) for p in pos])),
        # every third token sees nothing, or only the prefix
        "holes": dict(first_keys=i32([p + 1 if t % 3 == 0 else 0 for t, p in enumerate(pos)]),
                      prefix_lens=i32([5 * (b % 2) for b in range(len(lens))]), slopes=_slopes(hq)),
        "all": dict(soft_cap=30.0, slopes=_slopes(hq), window=150, prefix_lens=i32([min(n, 20) for n in lens]),
                    first_keys=i32([p // 90 * 90 for p in pos])),
    }
    return some[name]


def _check(a, rules, st=(0, -1), rows=None):
    out, lse = pa.paged_attention_scored(**a, **rules)
    got = pa.check_errors()
    assert got == st, got
    want, want_lse, tol, tol_lse = ref.attention(a["q"], a["k_cache"], a["v_cache"], a["block_tables"],
                                                 a["seq_lens"].tolist(), a["query_start_loc"].tolist(), a["scale"], **rules)
    keep = slice(None) if rows is None else rows
    o, l = out.double()[keep], lse.double()[keep]
    want, want_lse, tol, tol_lse = want[keep], want_lse[keep], tol[keep], tol_lse[keep]
    assert not o.isnan().any() and not l.isnan().any()
    empty = want_lse == -math.inf
    assert torch.equal(l == -math.inf, empty) and bool((o[empty] == 0).all())
    worst = ((o - want).abs() / tol).max().item()
    assert worst <= 1, ("out", worst)
    worst = ((l - want_lse).abs() / tol_lse)[~empty].max().item() if bool((~empty).any()) else 0.0
    assert worst <= 1, ("lse", worst)
    return out, lse


RULES = ["plain", "cap", "bias", "window", "window1", "sinks", "prefix", "docs", "holes", "all"]
HEADS = [(8, 2, 128), (4, 4, 128), (7, 1, 128), (16, 2, 256), (8, 1, 512)]
DECODE = [1, 15, 16, 17, 128, 129, 255, 257, 700, 2049]
MIXED = ([1, 16, 33, 130, 300, 515, 700, 64], [1, 16, 1, 130, 5, 257, 64, 0])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("rule", RULES)
def test_decode(rule, heads):
    a = _batch(DECODE, [1] * len(DECODE), *heads, seed=1, spread=3.0)
    _check(a, _rules(rule, DECODE, [1] * len(DECODE), heads[0]))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("rule", RULES)
def test_drafts(rule, heads):
    lens, new = [3, 18, 131, 260, 1030], [3, 2, 4, 1, 4]
    a = _batch(lens, new, *heads, seed=2, layout="head_major")
    _check(a, _rules(rule, lens, new, heads[0]))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("rule", RULES)
def test_mixed_chunks(rule, heads):
    a = _batch(*MIXED, *heads, seed=3, spread=2.0)
    _check(a, _rules(rule, *MIXED, heads[0]))


@pytest.mark.parametrize("heads", [(8, 2, 128), (32, 1, 128), (128, 1, 128), (6, 2, 256), (4, 1, 512)])
@pytest.mark.parametrize("rule", ["cap", "sinks", "docs", "all"])
@pytest.mark.parametrize("lens,new", [([1153], [1153]), ([1300], [129]), ([4171, 300], [40, 300])])
def test_prompts(rule, heads, lens, new):
    a = _batch(lens, new, *heads, seed=4)
    _check(a, _rules(rule, lens, new, heads[0]))


@pytest.mark.parametrize("n", [63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 383, 385])
def test_prompt_lengths_at_tile_edges(n):
    for heads in ((8, 2, 128), (4, 2, 256)):
        a = _batch([n, n // 2], [n, n // 2], *heads, seed=n)
        _check(a, _rules("cap", [n, n // 2], [n, n // 2], heads[0]))
        _check(a, dict(window=64, slopes=_slopes(heads[0])))


@pytest.mark.parametrize("new", [1, 7, 200])
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 256), (4, 1, 512)])
def test_pages_behind_a_window_may_be_anything(new, heads):
    lens = [600, 220, 1025]
    a = _batch(lens, [new] * 3, *heads, seed=5)
    for b, n in enumerate(lens):
        first = max(0, n - new + 1 - 50)  # the first key that some token sees
        a["block_tables"][b, :first // 16] = torch.tensor([POISON, -1, a["k_cache"].shape[0]], device="cuda",
                                                          dtype=torch.int32).repeat(30)[:first // 16]
    _check(a, dict(window=50))
    a = _batch(lens, [new] * 3, *heads, seed=5)
    for b, n in enumerate(lens):
        first = max(0, n - new + 1 - 50)
        a["block_tables"][b, 1:max(1, first // 16)] = -7
    _check(a, dict(window=50, prefix_lens=i32([16, 3, 9])))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("new,heads", [(1, (8, 2, 128)), (4, (8, 2, 128)), (4, (4, 1, 256)), (3, (4, 1, 512)),
                                       (300, (8, 2, 128)), (300, (4, 1, 256)), (40, (4, 1, 512))])
def test_hidden_keys_never_matter(value, which, new, heads):
    """Keys outside every row's window, and keys that only later tokens see."""
    lens = [640, 517]
    a = _batch(lens, [new] * 2, *heads, seed=6)
    rules = dict(window=200, soft_cap=0.0)
    hidden = torch.zeros(2 * new, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        spots = [n - new - 200, max(0, n - new - 230), 3] + ([n - 2] if new > 1 else [])
        for j in spots:
            a[which + "_cache"][int(a["block_tables"][b, j // 16]), j % 16] = value
        if new > 1:
            hidden[b * new + new - 2:(b + 1) * new] = True   # the last two tokens see key n - 2
    _check(a, rules, rows=~hidden)


def test_a_seen_nan_shows():
    lens, new = [300, 300], [300, 1]
    for which in "kv":
        a = _batch(lens, new, 8, 2, 128, seed=7)
        a[which + "_cache"][int(a["block_tables"][0, 6]), 4, 1] = math.nan     # key 100 of KV head 1
        out, lse = pa.paged_attention_scored(**a, window=50)
        bad = torch.zeros(301, dtype=torch.bool)
        bad[100:150] = True
        assert torch.equal(out[:, 4:].isnan().flatten(1).any(1).cpu(), bad)
        assert not out[:, :4].isnan().any()


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 256), (4, 1, 512)])
@pytest.mark.parametrize("new", [1, 5, 200])
def test_a_bad_page_makes_the_rows_that_see_it_nan(heads, new):
    for page in (-1, POISON, 10**6):
        lens = [700, 400]
        a = _batch(lens, [new, new], *heads, seed=8)
        a["block_tables"][0, 42] = page          # keys 672 .. 687
        out, lse = pa.paged_attention_scored(**a, window=30)
        assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 0)
        pos = torch.arange(700 - new, 700)
        bad = (pos >= 672) & (pos - 30 < 687)
        assert torch.equal(out[:new].isnan().flatten(1).all(1).cpu(), bad)
        assert torch.equal(lse[:new].isnan().all(1).cpu(), bad) and torch.equal(lse[:new].isnan().any(1).cpu(), bad)
        assert not out[new:].isnan().any()


def test_bad_requests_are_nan_and_others_intact():
    lens, new = [300, 200, 64], [5, 5, 5]
    for what in ("short", "past_row", "past_bound", "past_query_bound"):
        a = _batch(lens, new, 8, 2, 128, seed=9)
        if what == "short":
            a["seq_lens"][1] = 4
        elif what == "past_row":
            a["seq_lens"][1], a["max_seq_len"] = a["block_tables"].shape[1] * 16 + 1, 10**6
        elif what == "past_bound":
            a["max_seq_len"], a["seq_lens"][1] = 310, 311
        else:
            a["query_start_loc"] = i32([0, 5, 12, 15])
            a["seq_lens"][2] = 64
        out, lse = pa.paged_attention_scored(**a, window=90)
        assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 1)
        s, e = a["query_start_loc"].tolist()[1:3]
        assert out[s:e].isnan().all() and lse[s:e].isnan().all()
        assert not out[:s].isnan().any() and not out[e:].isnan().any()


def test_rows_of_no_request_and_empty_requests_are_left_alone():
    a = _batch([40, 0, 33], [2, 0, 3], 8, 2, 128, seed=10)
    q = torch.cat([a["q"], a["q"]])
    a["q"] = q
    out = torch.full_like(q.contiguous(), 7.0)
    lse = torch.full((10, 8), 7.0, device="cuda")
    pa.paged_attention_scored(**a, soft_cap=5.0, out=out, lse=lse)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert bool((out[5:] == 7).all()) and bool((lse[5:] == 7).all()) and not bool((out[:5] == 7).all(-1).any())
    for new, bounds in (([0], (0, 40)), ([0], (1, 40))):
        b = _batch([40], new, 8, 2, 128)
        b["q"], b["max_query_len"], b["max_seq_len"] = q[:1], *bounds
        o = torch.full((1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        pa.paged_attention_scored(**b, out=o)
        assert pa.check_errors() == (pa.PA_OK, -1) and bool((o == 7).all())


@pytest.mark.parametrize("new", [1, 300])
def test_loose_bounds_and_any_workspace(new):
    lens = [700, 333]
    a = _batch(lens, [new] * 2, 8, 2, 128, seed=11)
    rules = dict(soft_cap=10.0, window=400)
    _check(a, rules)
    a["max_seq_len"], a["max_query_len"] = 5000, new + 70
    n = pa.scored_workspace_size(2, 8, 2, 128, a["max_query_len"], 5000)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:]
    outs = [pa.paged_attention_scored(**a, **rules, workspace=ws)[0] for _ in range(2)]
    assert torch.equal(outs[0], outs[1])
    _check(a, rules)


def test_extreme_caps_scores_and_slopes():
    lens, new = [500, 129], [1, 129]
    a = _batch(lens, new, 8, 2, 128, seed=12, spread=200.0)      # scores of several hundred
    for rules in (dict(soft_cap=0.001), dict(soft_cap=2000.0), dict(soft_cap=50.0), {},
                  dict(slopes=torch.tensor([0, 1e-6, -0.02, 1, 30, 1000, -3, 0.5], device="cuda"))):
        _check(a, rules)


def test_a_prefix_far_behind_keeps_its_differences():
    """Rows that see only keys thousands of positions back: the bias's common part
    must not cost the keys' differences."""
    lens, new = [9000], [3]
    a = _batch(lens, new, 8, 2, 128, seed=13)
    rules = dict(first_keys=i32([8998, 8999, 9000]), prefix_lens=i32([300]), slopes=_slopes(8))
    _check(a, rules)


def test_against_the_plain_attention():
    a = _batch([513, 100], [200, 100], 8, 2, 128, seed=14)
    out, lse = pa.paged_attention(**a)
    mine, my_lse = pa.paged_attention_scored(**a)
    assert (lse - my_lse).abs().max() < 1e-4 and (out.float() - mine.float()).abs().max() < 2e-2
