"""pa_build_step_metadata on the GPU against a plain loop: every output equal,
everything not named as written left alone, in place and captured."""
import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import step_reference as ref

pytestmark = pytest.mark.gpu

POISON = 2**31 - 1


def _setup(ctx, new, pad=0, cols=None, spare=3, cursor=2, seed=0):
    rng = np.random.default_rng(seed)
    pages = lambda n: -(-max(n, 0) // 16)
    cols = cols or max([pages(c + q) for c, q in zip(ctx, new)] + [1])
    have = [min(pages(c), cols) for c in ctx]
    need = sum(max(0, pages(c + q) - pages(c)) for c, q in zip(ctx, new))
    blocks = sum(have) + need + spare + cursor + 4
    perm = rng.permutation(blocks).astype(np.int32)
    tables = np.full((len(ctx), cols), POISON, np.int32)
    at = 0
    for b, h in enumerate(have):
        tables[b, :h] = perm[at:at + h]
        at += h
    free = perm[at:at + cursor + need + spare].copy()
    return dict(ctx=list(ctx), new=list(new), tables=tables, free=free, cursor=cursor, num_blocks=blocks,
                num_tokens=max(0, sum(max(q, 0) for q in new)) + pad)


def _device(s):
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
    d = dict(context_lens=i32(s["ctx"]), query_lens=i32(s["new"]), block_tables=i32(s["tables"]),
             free_pages=i32(s["free"]), num_blocks=s["num_blocks"],
             slot_mapping=torch.full((s["num_tokens"],), -99, dtype=torch.int64, device="cuda"),
             positions=torch.full((s["num_tokens"],), -99, dtype=torch.int32, device="cuda"),
             seq_lens=i32([-99] * len(s["ctx"])), query_start_loc=i32([-99] * (len(s["ctx"]) + 1)),
             cursor_out=i32([-99]), cursor_in=i32([s["cursor"]]))
    return d


def _compare(d, s):
    want = ref.step_metadata(s["ctx"], s["new"], s["tables"], s["free"], s["cursor"], s["num_blocks"], s["num_tokens"])
    for name, w in zip(("block_tables", "slot_mapping", "positions", "seq_lens", "query_start_loc"), want):
        got = d[name].cpu().numpy()
        assert np.array_equal(got, w), (name, np.argwhere(got != w)[:4])
    assert int(d["cursor_out"]) == want[5]
    return want[6]


CASES = {
    "one_new_token": ([0], [1]),
    "page_ends": ([15, 16, 17, 31, 32, 0, 1], [1, 1, 1, 1, 1, 16, 15]),
    "idle_and_empty": ([0, 40, 0, 5, 100], [0, 0, 0, 3, 0]),
    "nothing_new": ([3, 0], [0, 0]),
    "mixed": ([0, 513, 1000, 4171, 7168, 31], [300, 1, 0, 257, 1, 17]),
    "b300": ([(37 * i) % 700 for i in range(300)], [(i * i) % 23 for i in range(300)]),
    "b1025": ([(11 * i) % 90 for i in range(1025)], [i % 3 for i in range(1025)]),
    "b8192": ([i % 50 for i in range(8192)], [1] * 8192),
    "long_prompt": ([0, 64], [70001, 1]),
}


@pytest.mark.parametrize("pad", [0, 37])
@pytest.mark.parametrize("case", list(CASES))
def test_matches_reference(case, pad):
    s = _setup(*CASES[case], pad=pad)
    d = _device(s)
    pa.build_step_metadata(**d)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _compare(d, s) is None


def test_no_cursor_no_tokens_and_exact_free_list():
    s = _setup([16, 7], [0, 0], cursor=0, spare=0)
    d = _device(s)
    d["cursor_in"] = None
    pa.build_step_metadata(**d)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _compare(d, s) is None
    s = _setup([16, 7], [17, 9], cursor=0, spare=0)   # takes the very last free page
    d = _device(s)
    d["cursor_in"] = None
    pa.build_step_metadata(**d)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _compare(d, s) is None and int(d["cursor_out"]) == len(s["free"])


def test_lengths_and_cursor_advance_in_place_in_a_graph():
    """A decode step whose graph advances its own lengths and cursor: ten
    replays equal ten steps of the reference."""
    ctx = [5, 15, 16, 40, 0]
    s = _setup(ctx, [10] * 5, spare=2, cursor=0)
    s["new"], s["num_tokens"] = [1] * 5, 8
    d = _device(s)
    d["seq_lens"], d["cursor_out"] = d["context_lens"], d["cursor_in"]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.init()
    call = pa.prepare_build_step_metadata(**d, stream=st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for _ in range(10):
        g.replay()
        torch.cuda.synchronize()
        assert _compare(d, s) is None
        w = ref.step_metadata(s["ctx"], s["new"], s["tables"], s["free"], s["cursor"], s["num_blocks"], 8)
        s["tables"], s["ctx"], s["cursor"] = w[0], w[3].tolist(), w[5]
    assert pa.check_errors() == (pa.PA_OK, -1)


@pytest.mark.parametrize("what", ["negative_ctx", "negative_new", "too_long", "ctx_past_table"])
def test_bad_request_brings_nothing(what):
    ctx, new = [20, 33, 8], [5, 2, 30]
    if what == "negative_ctx":
        ctx[1] = -4
    elif what == "negative_new":
        new[1] = -1
    elif what == "too_long":
        new[1] = 100
    else:
        ctx[1] = 2**31 - 1
    s = _setup(ctx, new, cols=4, pad=3)
    d = _device(s)
    pa.build_step_metadata(**d)
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 1)
    assert _compare(d, s) == ("request", 1)


def test_bad_page_ids_give_no_slots():
    s = _setup([20, 33], [40, 2])
    s["free"][3] = s["num_blocks"]          # a new page outside the pool
    s["tables"][1, 2] = -5                   # the page that token 33 goes to
    d = _device(s)
    pa.build_step_metadata(**d)
    st, idx = pa.check_errors()
    assert st == pa.PA_ERR_BAD_METADATA and idx in (0, 1)
    assert _compare(d, s) is not None


@pytest.mark.parametrize("what", ["pages", "tokens", "cursor_low", "cursor_high"])
def test_step_that_does_not_fit_is_empty(what):
    s = _setup([20, 33, 0], [40, 2, 16], cursor=2, spare=0)
    want = (pa.PA_ERR_BAD_METADATA, 3)
    if what == "pages":
        s["free"] = s["free"][:-1]
        want = (pa.PA_ERR_WORKSPACE, 3)   # (4 - 2) + (3 - 3) + (1 - 0) pages
    elif what == "tokens":
        s["num_tokens"] -= 1
    else:
        s["cursor"] = -1 if what == "cursor_low" else len(s["free"]) + 1
    d = _device(s)
    pa.build_step_metadata(**d)
    assert pa.check_errors() == want
    assert _compare(d, s) is not None
    assert int(d["query_start_loc"].abs().sum()) == 0 and bool((d["slot_mapping"] == -1).all())
