"""pa_paged_attention_scored as programs call it: captured and replayed, on other
streams, beside another call, into pinned memory, far into a large pool, with
many requests, and in a row with forks, writes, releases and compactions."""
import math

import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import score_reference as ref
from tests.test_gpu_scored_attention import _batch, _check, _rules, _slopes, i32

pytestmark = pytest.mark.gpu


def _results(a):
    T, hq, dh = a["q"].shape
    return (torch.empty(T, hq, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(T, hq, device="cuda"))


def _workspace(a, **kw):
    hq, dh = a["q"].shape[1:]
    return pa.new_scored_workspace(a["seq_lens"].numel(), hq, a["k_cache"].shape[2], dh, a["max_query_len"],
                                   a["max_seq_len"], **kw)


def _prepare(a, rules, ws, stream=None):
    out, lse = _results(a)
    return pa.prepare_paged_attention_scored(**a, out=out, lse=lse, workspace=ws, stream=stream, **rules), out, lse


def _same(a, rules, out, lse):
    """Bitwise what a call by itself gives, which is right."""
    want, want_lse = _check(a, rules)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


DECODE = ([700, 33, 1, 260], [1, 1, 1, 1], 8, 2, 128)
PROMPT = ([300, 513, 40], [300, 200, 40], 8, 2, 128)
WIDE = ([600, 70], [600, 3], 4, 1, 512)


def test_a_captured_call_follows_its_inputs():
    """A replay reads lengths, tables, rules and rows as they are then."""
    for shape in (DECODE, PROMPT, WIDE):
        a = _batch(*shape, seed=1)
        lens, new, hq = shape[:3]
        rules = dict(soft_cap=30.0, slopes=_slopes(hq), window=90, prefix_lens=i32([3] * len(lens)),
                     first_keys=i32([0] * sum(new)))
        st = torch.cuda.Stream()
        call, out, lse = _prepare(a, rules, _workspace(a), st)
        pa.init()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        for turn in range(4):
            if turn == 1:
                a["q"].mul_(2)
                rules["slopes"].mul_(0.5)
            if turn == 2:
                rules["first_keys"].fill_(20)
                rules["prefix_lens"].zero_()
            if turn == 3:
                a["seq_lens"].sub_(i32([n > x for n, x in zip(lens, new)]))
            g.replay()
            torch.cuda.synchronize()
            _same(a, rules, out, lse)


def test_two_captured_graphs_share_a_workspace():
    """Calls of other bounds, kernels and head layouts in one workspace: each
    replay writes all of what it reads there."""
    shapes = [DECODE, PROMPT, WIDE, ([513] * 3, [2] * 3, 16, 2, 256)]
    batches = [_batch(*s, seed=i) for i, s in enumerate(shapes)]
    rules = [dict(soft_cap=20.0), dict(window=64), {}, dict(slopes=_slopes(16))]
    ws = max((_workspace(a) for a in batches), key=lambda t: t.numel())
    ws.fill_(0xFF)
    st = torch.cuda.Stream()
    pa.init()
    graphs = []
    for a, r in zip(batches, rules):
        call, out, lse = _prepare(a, r, ws, st)
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            call()
        graphs.append((g, out, lse))
    with torch.cuda.stream(st):
        for order in ([0, 1, 2, 3], [3, 1, 0, 2], [2, 0, 2, 1, 3]):
            for g, out, lse in graphs:
                out.fill_(7.0)
                lse.fill_(7.0)
            for i in order:
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for a, r, (g, out, lse) in zip(batches, rules, graphs):
        _same(a, r, out, lse)


def test_on_another_stream_behind_its_producer():
    a, side = _batch(*PROMPT, seed=3), torch.cuda.Stream()
    q = a["q"].clone()
    torch.cuda.synchronize()
    ws = _workspace(a)
    call, out, lse = _prepare(a, dict(window=100), ws, side)
    with torch.cuda.stream(side):
        a["q"].zero_()
        for _ in range(20):
            a["q"].add_(q * 0.05)
        a["q"].copy_(q)
        call()
    side.synchronize()
    _same(a, dict(window=100), out, lse)


def test_calls_beside_one_another():
    """Two streams, each with a workspace of its own."""
    batches = [_batch(*PROMPT, seed=4), _batch(*DECODE, seed=5)]
    rules = [dict(soft_cap=25.0), dict(window=200)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = [_prepare(a, r, _workspace(a), s) for a, r, s in zip(batches, rules, streams)]
    torch.cuda.synchronize()
    for _ in range(20):
        for call, _, _ in calls:
            call()
    torch.cuda.synchronize()
    for a, r, (_, out, lse) in zip(batches, rules, calls):
        _same(a, r, out, lse)


@pytest.mark.parametrize("shape", [DECODE, PROMPT, WIDE])
def test_results_in_pinned_memory(shape):
    a = _batch(*shape, seed=6)
    out, lse = (t.cpu().pin_memory() for t in _results(a))
    pa.paged_attention_scored(**a, out=out, lse=lse, workspace=_workspace(a), window=77)
    torch.cuda.synchronize()
    _same(a, dict(window=77), out.cuda(), lse.cuda())


@pytest.mark.parametrize("shape", [DECODE, PROMPT, WIDE])
def test_without_lse_and_with_a_larger_workspace(shape):
    a = _batch(*shape, seed=7)
    ws = torch.full((_workspace(a).numel() + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = pa.paged_attention_scored(**a, want_lse=False, workspace=ws)
    assert lse is None and torch.equal(out, _check(a, {})[0])


@pytest.mark.parametrize("dh,hkv", [(128, 1), (512, 2)])
@pytest.mark.parametrize("new", [1, 150])
def test_pages_past_32_bit_offsets(dh, hkv, new):
    """The pool's last pages, whose elements lie past 2^32; a row whose sum
    overflows takes the path key by key there too."""
    stride = 2 * 16 * hkv * dh
    nb = 2**32 // stride + 40
    pool = torch.empty(nb, 2, 16, hkv, dh, dtype=torch.bfloat16, device="cuda")
    pool[-30:] = torch.randn(30, 2, 16, hkv, dh, device="cuda").to(torch.bfloat16)
    pool[0].fill_(math.nan)
    n, hq = 330, 4 * hkv
    tables = torch.arange(nb - 1, nb - 22, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    a = dict(q=torch.randn(new, hq, dh, device="cuda").to(torch.bfloat16), k_cache=pool[:, 0], v_cache=pool[:, 1],
             block_tables=tables, seq_lens=i32([n]), query_start_loc=i32([0, new]), scale=dh**-0.5, max_query_len=new,
             max_seq_len=n)
    _check(a, dict(window=200, prefix_lens=i32([5])))
    # a value past BF16's range seen by all: its column is infinite, the others are right
    pool[nb - 1, 1, 3, :, 0] = math.inf
    out, _ = pa.paged_attention_scored(**a)
    assert bool((out[..., 0] == math.inf).all()) and bool(out[..., 1:].isfinite().all())
    pool[nb - 1, 1, 3, :, 0] = 0
    want, _ = _check(a, {})
    err = (out[..., 1:].double() - want[..., 1:].double()).abs()
    # (both are within 2^-8 and the probabilities' 2^-8 of the true value)
    assert bool((err <= 2.0**-6 * (want[..., 1:].double().abs() + 1)).all())


@pytest.mark.parametrize("shape,count", [((4, 2, 128), 8192), ((2, 1, 256), 3000)])
def test_many_requests(shape, count):
    hq, hkv, dh = shape
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(1, 60, (count,), generator=g).tolist()
    for new in ([1] * count, [min(n, 1 + 30 * (b % 50 == 0)) for b, n in enumerate(lens)]):
        if max(new) > 1 and count > 3000:
            continue
        a = _batch(lens, new, hq, hkv, dh, seed=9)
        rules = dict(soft_cap=15.0, window=20)
        out, lse = pa.paged_attention_scored(**a, **rules)
        assert pa.check_errors() == (0, -1)
        starts = a["query_start_loc"].tolist()
        for b in list(range(0, count, 97)) + [count - 1]:
            rows = slice(starts[b], starts[b + 1])
            want, want_lse, tol, tol_lse = ref.attention(
                a["q"][rows], a["k_cache"], a["v_cache"], a["block_tables"][b:b + 1], [lens[b]], [0, new[b]], a["scale"],
                **rules)
            assert bool(((out[rows].double() - want).abs() <= tol).all()), b
            assert bool(((lse[rows].double() - want_lse).abs() <= tol_lse).all()), b
        assert bool(out.isfinite().all()) and bool(lse.isfinite().all())


@pytest.mark.parametrize("hq,hkv", [(128, 1), (32, 1), (33, 1), (96, 3), (16, 16)])
def test_group_sizes(hq, hkv):
    for lens, new in (([200, 17], [1, 1]), ([200, 90], [3, 90])):
        a = _batch(lens, new, hq, hkv, 128, seed=10)
        _check(a, _rules("all", lens, new, hq))


@pytest.mark.parametrize("hq,hkv,dh", [(3, 1, 512), (5, 1, 256), (12, 4, 512)])
def test_groups_that_do_not_divide_a_tile(hq, hkv, dh):
    lens, new = [300, 90, 43], [300, 1, 43]
    a = _batch(lens, new, hq, hkv, dh, seed=14)
    for rule in ("cap", "all"):
        _check(a, _rules(rule, lens, new, hq))


@pytest.mark.parametrize("hq,hkv,dh", [(8, 2, 128), (6, 2, 256), (4, 1, 512)])
@pytest.mark.parametrize("new", [1, 20, 300])
def test_nothing_to_see(hq, hkv, dh, new):
    """Tokens whose documents begin behind them, beside some that see keys, and alone."""
    lens, n = [300, 310, 1000], [new, new, min(new, 3)]
    a = _batch(lens, n, hq, hkv, dh, seed=15)
    pos = [L - x + i for L, x in zip(lens, n) for i in range(x)]
    first = [p + 1 for p in pos]
    out, lse = _check(a, dict(first_keys=i32(first)))
    assert not out.any() and bool((lse == -math.inf).all())
    first[new:2 * new] = [0] * new
    _check(a, dict(first_keys=i32(first), soft_cap=30.0))
    _check(a, dict(first_keys=i32([2**31 - 1] * len(pos)), prefix_lens=i32([0, 0, 7])))


@pytest.mark.parametrize("bound", [4, 300])
def test_tokens_of_no_request(bound):
    a = _batch([300, 40], [3, 1], 8, 2, 128, seed=16)
    a.update(query_start_loc=i32([0, 0, 0]), max_query_len=bound)
    out, lse = torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 8), 7.0, device="cuda")
    pa.paged_attention_scored(**a, out=out, lse=lse)
    assert pa.check_errors() == (0, -1) and bool((out == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("new", [4, 300])
def test_decreasing_query_starts_touch_nothing_else(new):
    """Requests that claim the same rows, and ones that end before they begin."""
    a = _batch([400] * 5, [new, 0, 0, 0, 0], 8, 2, 128, seed=17)
    a["query_start_loc"] = i32([0, new, 0, new, 0, new])
    out = torch.full((new + 2, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((new + 2, 8), 7.0, device="cuda")
    pa.paged_attention_scored(**a, out=out[1:-1], lse=lse[1:-1])
    assert pa.check_errors()[0] == pa.PA_ERR_BAD_METADATA
    for t in (out, lse):
        assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all())


def test_pages_shared_and_held_twice():
    """Requests that share pages, and a table that names one page twice."""
    for new in (1, 40):
        a = _batch([200, 200], [new] * 2, 8, 2, 128, seed=11)
        a["block_tables"][1, :9] = a["block_tables"][0, :9]
        a["block_tables"][1, 4] = a["block_tables"][1, 2]
        _check(a, dict(window=150, slopes=_slopes(8)))


def test_the_same_result_every_time():
    a = _batch([3000, 900, 1700], [700, 900, 1], 8, 2, 128, seed=12)
    for rules in ({}, dict(soft_cap=20.0), dict(slopes=_slopes(8))):
        first = pa.paged_attention_scored(**a, **rules)
        for _ in range(5):
            again = pa.paged_attention_scored(**a, **rules)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_model_with_windows_serves_forked_requests():
    """A prompt, three continuations of it, four steps of each with layers of two
    kinds (window and first tokens; capped), pages behind the window released from
    the windowed layer's tables, a compaction: every step matches the reference
    on the tokens written."""
    hq, hkv, dh, window, sinks = 8, 2, 128, 48, 4
    g = torch.Generator(device="cuda").manual_seed(13)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    nb, cols, reqs, n0 = 80, 12, 4, 100
    pools = [torch.full((nb, 2, 16, hkv, dh), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    caches = [(p[:, 0], p[:, 1]) for p in pools]
    tables = torch.full((reqs, cols), -1, dtype=torch.int32, device="cuda")
    shares, free, cursor = i32([0] * nb), i32(torch.randperm(nb).tolist()), i32([0])
    lens = i32([0] * reqs)
    layers = [dict(window=window, prefix_lens=i32([sinks] * reqs)), dict(soft_cap=20.0)]
    written = [[[], []] for _ in range(reqs)]  # [request][layer]: K, V rows

    def step(new):
        total = sum(new)
        slots, pos, start = torch.zeros(total, dtype=torch.int64, device="cuda"), i32([0] * total), i32([0] * (reqs + 1))
        pa.build_step_metadata(lens, i32(new), tables, free, nb, slots, pos, lens, start, cursor, cursor)
        starts = start.tolist()
        for layer, (k, v) in enumerate(caches):
            kn, vn = rnd(total, hkv, dh), rnd(total, hkv, dh)
            pa.reshape_and_cache(kn, vn, k, v, slots)
            for b in range(reqs):
                if new[b]:
                    written[b][layer] = written[b][layer] + [(kn[starts[b]:starts[b + 1]], vn[starts[b]:starts[b + 1]])]
            q = rnd(total, hq, dh)
            # the window's layer holds no page behind its window and the first tokens
            t = tables.clone()
            if layer == 0:
                for b, n in enumerate(lens.tolist()):
                    if new[b]:
                        t[b, 1:max(n - new[b] - window + 1, 0) // 16] = 2**30
            out, lse = pa.paged_attention_scored(q, k, v, t, lens, start, dh**-0.5, max(new), cols * 16, **layers[layer])
            assert pa.check_errors() == (0, -1)
            for b in range(reqs):
                if not new[b]:
                    continue
                rows = slice(starts[b], starts[b + 1])
                kk, vv = (torch.cat([w[i] for w in written[b][layer]]) for i in (0, 1))
                n = kk.shape[0]
                fill = lambda x: torch.cat([x, x.new_zeros(-n % 16, hkv, dh)]).view(-1, 16, hkv, dh)
                rules = {key: x[b:b + 1] if key == "prefix_lens" else x for key, x in layers[layer].items()}
                want, want_lse, tol, tol_lse = ref.attention(
                    q[rows], fill(kk), fill(vv), torch.arange(-(-n // 16), device="cuda")[None], [n], [0, new[b]], dh**-0.5,
                    **rules)
                assert bool(((out[rows].double() - want).abs() <= tol).all()), (layer, b)
                assert bool(((lse[rows].double() - want_lse).abs() <= tol_lse).all()), (layer, b)

    step([n0, 0, 0, 0])
    src, dst = i32([0] * 3), i32([0] * 3)
    pa.fork_requests(i32([0, 0, 0]), i32([1, 2, 3]), i32([n0, n0 - 5, 64]), lens, tables, shares, shares, free, cursor, cursor,
                     lens, src, dst)
    pa.copy_pages(caches, src, dst)
    for b, n in ((1, n0), (2, n0 - 5), (3, 64)):
        for layer in range(2):
            k, v = written[0][layer][0]
            written[b][layer] = [(k[:n], v[:n])]
    step([1, 1, 1, 1])
    step([1, 5, 1, 40])
    # request 1's last two tokens are rejected, request 0 ends
    keep = lens.clone()
    keep[0], keep[1] = 0, keep[1] - 2
    pa.release_pages(lens, keep, tables, shares, shares, free, cursor, cursor, lens)
    written[0] = [[], []]
    for layer in range(2):
        k, v = (torch.cat([w[i] for w in written[1][layer]])[:-2] for i in (0, 1))
        written[1][layer] = [(k, v)]
    assert pa.check_errors() == (0, -1)
    step([0, 1, 1, 1])
    src, dst, counts = i32([0] * nb), i32([0] * nb), i32([0, 0])
    pa.compact_pages(lens, tables, tables, shares, shares, free, cursor, cursor, src, dst, counts)
    pa.copy_pages(caches, src, dst)
    assert pa.check_errors() == (0, -1) and int(cursor) == int(counts[0])
    step([20, 1, 1, 1])
    step([1, 1, 1, 1])
