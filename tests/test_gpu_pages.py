"""Copies of pages, forks, releases and compactions on the GPU against plain
loops: every output equal, everything not named as written left alone, in place,
captured, and the errors."""
import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import page_reference as ref

pytestmark = pytest.mark.gpu

POISON = 2**31 - 1
i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")


# ------------------------------------------------------------------- copies --

def _pools(layout, layers, nb, hkv, dh, seed=0):
    """`layers` (k, v) views [nb, 16, hkv, dh] and the tensors they lie in."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = lambda *shape: torch.randint(-2**15, 2**15, shape, generator=g, device="cuda", dtype=torch.int16)
    out, owners = [], []
    for _ in range(layers):
        if layout == "interleaved":
            t = bits(nb, 2, 16, hkv, dh)
            kv = (t[:, 0], t[:, 1])
        elif layout == "separate":
            t = bits(2, nb, 16, hkv, dh)
            kv = (t[0], t[1])
        elif layout == "head_major":
            t = bits(nb, 2, hkv, 16, dh)
            kv = (t[:, 0].transpose(1, 2), t[:, 1].transpose(1, 2))
        elif layout == "heads_outermost":
            t = bits(2, hkv, nb, 16, dh)
            kv = (t[0].permute(1, 2, 0, 3), t[1].permute(1, 2, 0, 3))
        elif layout == "some_heads":
            t = bits(nb, 2, 16, hkv + 2, dh)
            kv = (t[:, 0, :, 1:1 + hkv], t[:, 1, :, 1:1 + hkv])
        else:  # padded rows, every other head
            t = bits(nb, 2, 16, 2 * hkv, dh + 8)
            kv = (t[:, 0, :, ::2, :dh], t[:, 1, :, ::2, :dh])
        out.append(tuple(x.view(torch.bfloat16) for x in kv))
        owners.append(t)
    return out, owners


@pytest.mark.parametrize("layout", ["interleaved", "separate", "head_major", "heads_outermost", "some_heads", "padded"])
@pytest.mark.parametrize("hkv,dh,layers", [(1, 128, 1), (2, 128, 3), (3, 256, 2), (2, 512, 1)])
def test_copy_pages(layout, hkv, dh, layers):
    nb, n = 41, 13
    caches, owners = _pools(layout, layers, nb, hkv, dh)
    order = np.random.default_rng(dh + hkv).permutation(nb).astype(np.int32)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    src[4] = -1                 # padding
    src[7], dst[8] = dst[7], src[8]   # onto itself
    want = [t.clone() for t in owners]
    for (k, v), t, w in zip(caches, owners, want):
        for view in (k, v):
            x = torch.as_strided(w.view(torch.bfloat16), view.shape, view.stride(), view.storage_offset())
            for s, d in zip(src, dst):
                if s >= 0:
                    x[d] = x[s].clone()
    pa.copy_pages(caches, i32(src), i32(dst))
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert all(torch.equal(t, w) for t, w in zip(owners, want))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("hkv,dh,layers", [(1, 128, 2), (3, 128, 1), (2, 256, 3), (1, 512, 1)])
def test_copy_pages_quant(interleaved, hkv, dh, layers):
    nb, n = 30, 11
    g = torch.Generator(device="cuda").manual_seed(dh)
    shape = (nb, 2, hkv, 9 * dh) if interleaved else (2, nb, hkv + 1, 9 * dh)
    owners = [torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(layers)]
    views = [(t[:, 0], t[:, 1]) if interleaved else (t[0, :, :hkv], t[1, :, :hkv]) for t in owners]
    caches = [pa.QuantCache(k, v, dh, 0.5, 2.0) for k, v in views]
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    src, dst = order[:n].contiguous(), order[n:2 * n].contiguous()
    want = [t.clone() for t in owners]
    for w in want:
        for x in ((w[:, 0], w[:, 1]) if interleaved else (w[0, :, :hkv], w[1, :, :hkv])):
            x[dst.long()] = x[src.long()]
    pa.copy_pages_quant(caches, src, dst)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert all(torch.equal(t, w) for t, w in zip(owners, want))


@pytest.mark.parametrize("src,dst", [(7, 40), (40, 7), (2**31 - 1, 3), (3, 2**31 - 1), (3, -1), (5, -2**31)])
def test_copy_pages_outside_the_pool(src, dst):
    caches, owners = _pools("interleaved", 2, 40, 2, 128)
    want = [t.clone() for t in owners]
    for w in want:
        w[9] = w[1]
    pa.copy_pages(caches, i32([1, src]), i32([9, dst]))
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 1)
    assert all(torch.equal(t, w) for t, w in zip(owners, want))


def test_copy_pages_past_32_bit_offsets_and_nothing_to_do():
    nb = 300000                                   # 4.9 GB
    pool = torch.zeros((nb, 2, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    k, v = pool[:, 0], pool[:, 1]
    pool[17].normal_()
    pool[nb - 2].normal_()
    a, b = pool[17].clone(), pool[nb - 2].clone()
    pa.copy_pages([(k, v)], i32([17, nb - 2]), i32([nb - 1, 5]))
    pa.copy_pages([(k, v)], i32([]), i32([]))
    pa.copy_pages([], i32([1]), i32([2]))
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert torch.equal(pool[nb - 1], a) and torch.equal(pool[5], b) and int(pool[6:17].count_nonzero()) == 0


# -------------------------------------------------------------------- state --

class State:
    """Requests with shuffled, partly shared pages, and a free stack of all others."""

    def __init__(self, ctx, spare=20, cols=None, groups=1, common=0, seed=0, below=3):
        rng = np.random.default_rng(seed)
        cols = cols or max([ref.pages(c) for c in ctx] + [1]) + 1
        own = [ref.pages(c) - (common if c else 0) for c in ctx]
        heads = -(-len(ctx) // groups) * common
        used = sum(own) + heads
        self.num_blocks = used + spare
        perm = rng.permutation(self.num_blocks).astype(np.int32)
        self.tables = np.full((len(ctx), cols), POISON, np.int32)
        self.shares = np.zeros(self.num_blocks, np.int32)
        at = heads
        for b, c in enumerate(ctx):
            if c:
                head = perm[b // groups * common:b // groups * common + common]
                self.tables[b, :common] = head
                self.shares[head] += 1
                self.tables[b, common:common + own[b]] = perm[at:at + own[b]]
                at += own[b]
        self.shares[perm[:heads]] = np.maximum(self.shares[perm[:heads]] - 1, 0)
        self.free = np.full(self.num_blocks, -9, np.int32)
        self.cursor = used
        self.free[used:] = perm[used:]
        self.ctx = list(ctx)

    def device(self, in_place=False):
        d = dict(context_lens=i32(self.ctx), block_tables=i32(self.tables), shares_in=i32(self.shares),
                 free_pages=i32(self.free), cursor_in=i32([self.cursor]))
        d["shares_out"] = d["shares_in"] if in_place else torch.full_like(d["shares_in"], -77)
        d["cursor_out"] = d["cursor_in"] if in_place else i32([-77])
        return d


def _same(d, **want):
    for name, w in want.items():
        got = d[name].cpu().numpy()
        assert np.array_equal(got, np.asarray(w).reshape(got.shape)), (name, np.argwhere(got != w)[:4])


def _verdict(bad):
    """What check_errors has to say (the index of one of several bad items may be any of them)."""
    if bad is None:
        return pa.PA_OK
    return pa.PA_ERR_WORKSPACE if bad[0] in ("pages", "moves") else pa.PA_ERR_BAD_METADATA


# --------------------------------------------------------------------- fork --

def _fork(s, parents, children, lens, in_place):
    d = s.device(in_place)
    d["seq_lens"] = d["context_lens"] if in_place else torch.full_like(d["context_lens"], -77)
    d["copy_src"], d["copy_dst"] = i32([-77] * len(parents)), i32([-77] * len(parents))
    pa.fork_requests(parents=i32(parents), children=i32(children), fork_lens=None if lens is None else i32(lens), **d)
    st, idx = pa.check_errors()
    tables, shares, out, cursor, src, dst, bad = ref.fork(parents, children, lens, s.ctx, s.tables, s.shares, s.free,
                                                          s.cursor, s.num_blocks)
    _same(d, block_tables=tables, shares_out=shares, seq_lens=out, cursor_out=[cursor], copy_src=src, copy_dst=dst,
          free_pages=s.free)
    assert st == _verdict(bad)
    return idx, bad


FORKS = {
    "one": ([40], [0], None),
    "page_ends": ([15, 16, 17, 32, 1], [0, 1, 2, 3, 4], None),
    "nothing": ([0, 64], [0, 1, 1], [0, 0, 16]),
    "many_ways": ([1000], [0] * 70, None),
    "b300": ([(37 * i) % 900 for i in range(300)], list(range(300)) + list(range(0, 300, 7)), "cut"),
    "long": ([70001, 20], [0, 1, 0], [70001, 3, 69999]),
    "b4000": ([i % 50 for i in range(4000)], list(range(4000)), None),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", list(FORKS))
def test_fork(case, in_place):
    ctx, parents, lens = FORKS[case]
    if lens == "cut":
        lens = [max(0, ctx[p] - (5 * i) % 40) for i, p in enumerate(parents)]
    n = len(ctx)
    s = State(ctx + [0] * len(parents), spare=len(parents) + 2)
    _, bad = _fork(s, parents, [n + i for i in range(len(parents))], lens, in_place)
    assert bad is None


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what", ["parent", "parent_low", "child", "child_low", "child_used", "same_child", "too_long",
                                  "negative", "child_is_parent"])
def test_a_bad_fork_does_nothing(what, in_place):
    parents, children, lens = [0, 1, 0], [2, 3, 4], [30, 20, 17]
    s = State([40, 33, 0, 0, 0, 0])
    if what == "parent":
        parents[1] = 6
    elif what == "parent_low":
        parents[1] = -1
    elif what == "child":
        children[1] = 6
    elif what == "child_low":
        children[1] = -2**31
    elif what == "child_used":
        children[1] = 0
    elif what == "same_child":
        children[1] = 2
    elif what == "too_long":
        lens[1] = 34
    elif what == "negative":
        lens[1] = -1
    else:
        parents[1] = children[1] = 1
    idx, bad = _fork(s, parents, children, lens, in_place)
    assert bad == ("fork", 1) and idx == 1


def test_fork_context_past_the_row_and_bad_pages():
    s = State([40, 33, 0, 0], cols=4)
    s.ctx[1] = 65
    assert _fork(s, [0, 1], [2, 3], None, False) == (1, ("fork", 1))
    for page in (-1, 10**6, POISON):
        s = State([40, 33, 0, 0])
        s.tables[1, 0] = page                     # a whole page
        assert _fork(s, [0, 1], [2, 3], None, False) == (1, ("fork", 1))
        s = State([40, 33, 0, 0])
        s.tables[1, 2] = page                     # the partial one
        assert _fork(s, [0, 1], [2, 3], None, False) == (1, ("fork", 1))
        s = State([40, 33, 0, 0])
        s.free[s.cursor + 1] = page               # the new one
        assert _fork(s, [0, 1], [2, 3], None, False) == (1, ("fork", 1))


@pytest.mark.parametrize("in_place", [False, True])
def test_forks_that_do_not_fit(in_place):
    s = State([40, 33, 16, 0, 0, 0], spare=1)
    assert _fork(s, [0, 1, 2], [3, 4, 5], None, in_place) == (2, ("pages", 2))
    for cursor in (-1, s.num_blocks + 1):
        s.cursor = cursor
        assert _fork(s, [0, 1, 2], [3, 4, 5], None, in_place) == (3, ("call",))
    assert _fork(State([40]), [], [], None, in_place)[1] is None


# ------------------------------------------------------------------ release --

def _release(s, keep, in_place, loose=False):
    d = s.device(in_place)
    d["seq_lens"] = d["context_lens"] if in_place else torch.full_like(d["context_lens"], -77)
    pa.release_pages(keep_lens=i32(keep), **d)
    st, idx = pa.check_errors()
    shares, free, out, cursor, bad = ref.release(s.ctx, keep, s.tables, s.shares, s.free, s.cursor, s.num_blocks)
    if loose:  # the order of the freed pages is not named
        got = d["free_pages"].cpu().numpy()
        assert sorted(got[cursor:s.cursor]) == sorted(free[cursor:s.cursor]) and int(d["cursor_out"]) == cursor
        free[cursor:s.cursor] = got[cursor:s.cursor]
    _same(d, shares_out=shares, free_pages=free, seq_lens=out, cursor_out=[cursor], block_tables=s.tables)
    assert st == _verdict(bad)
    return idx, bad


RELEASES = {
    "one": ([40], [0], {}),
    "nothing": ([40, 0, 16], [40, 0, -1], {}),
    "page_ends": ([15, 16, 17, 33, 32, 48], [0, 15, 16, 32, 16, 17], {}),
    "drafts": ([7168, 7168, 4171, 513] * 16, [7165, 7163, 4167, 511] * 16, {}),
    "shared": ([200, 180, 150, 90] * 3, [0, 180, 0, 70, 0, 0, 0, 0, 160, 150, 0, 64], dict(groups=4, common=4)),
    "all_shared": ([700] * 40, [0] * 40, dict(groups=40, common=43)),
    "b300": ([(37 * i) % 900 + 64 for i in range(300)], None, dict(groups=5, common=4)),
    "b8192": ([i % 50 for i in range(8192)], [0] * 8192, {}),
    "long": ([70001, 20, 131072], [16, 20, 0], {}),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", list(RELEASES))
def test_release(case, in_place):
    ctx, keep, kw = RELEASES[case]
    if keep is None:
        keep = [0 if i % 3 == 0 else max(64, c - (7 * i) % 60) for i, c in enumerate(ctx)]
    _, bad = _release(State(ctx, **kw), keep, in_place)
    assert bad is None


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("what", ["negative_context", "past_row", "too_long", "shared_end", "bad_end"])
def test_a_bad_release_does_nothing(what, in_place):
    s, keep = State([100, 90, 80], groups=3, common=3, cols=8), [0, 50, 64]
    if what == "negative_context":
        s.ctx[1] = -5
    elif what == "past_row":
        s.ctx[1] = 129
    elif what == "too_long":
        keep[1] = 91
    elif what == "shared_end":
        keep[1] = 40
    else:
        s.tables[1, 3] = s.num_blocks
    assert _release(s, keep, in_place) == (1, ("request", 1))


def test_release_passes_over_bad_pages_and_frees_a_page_once():
    for page in (-3, 10**7):
        s = State([100, 90])
        s.tables[1, 4] = page
        assert _release(s, [0, 0], False) == (1, ("request", 1))
    s = State([100, 90])
    s.tables[1, 4] = s.tables[1, 3]           # the same index twice: given up once too often
    assert _release(s, [0, 0], False, loose=True) == (1, ("request", 1))


@pytest.mark.parametrize("in_place", [False, True])
def test_releases_that_do_not_fit(in_place):
    s = State([100, 90, 64], groups=3, common=2)
    s.cursor = 6
    assert _release(s, [0, 0, 0], in_place) == (13, ("pages", 13))  # 7 + 6 + 4 pages, two of them shared by all three
    for cursor in (-1, s.num_blocks + 1):
        s.cursor = cursor
        assert _release(s, [0, 0, 0], in_place) == (3, ("call",))


@pytest.mark.parametrize("in_place", [False, True])
def test_release_of_more_references_than_registers_hold(in_place):
    """180000 references, some to pages that two of the requests share."""
    s = State([360000] * 8, groups=2, common=1500, cols=22501)
    keep = [0, 0, 16 * 1499 + 16, 0, -1, 0, 100000, 0]
    _release(s, keep, in_place)
    s = State([360000] * 8, groups=2, common=1500, cols=22501, seed=1)
    _release(s, [0] * 8, in_place)


# --------------------------------------------------------------- compaction --

def _compact(s, max_moves, in_place, free_more=0):
    s.free = np.concatenate([np.full(free_more, -4, np.int32), s.free])
    s.cursor += free_more
    d = s.device(in_place)
    d["tables_out"] = d["block_tables"] if in_place else torch.full_like(d["block_tables"], -77)
    d["copy_src"], d["copy_dst"] = i32([-77] * max_moves), i32([-77] * max_moves)
    d["counts"] = i32([-77, -77])
    pa.compact_pages(**d)
    st, idx = pa.check_errors()
    tables, shares, free, cursor, src, dst, counts, bad = ref.compact(s.ctx, s.tables, s.shares, s.free, s.cursor,
                                                                      s.num_blocks, max_moves)
    if not in_place:
        left = np.ones_like(tables, bool)
        for b, c in enumerate(s.ctx):
            if 0 <= c <= tables.shape[1] * 16:
                left[b, :ref.pages(c)] = False
        tables[left] = -77
    _same(d, tables_out=tables, shares_out=shares, free_pages=free, cursor_out=[cursor], copy_src=src, copy_dst=dst,
          counts=counts)
    assert st == _verdict(bad)
    return idx, bad


COMPACTIONS = {
    "one": dict(ctx=[40]),
    "empty": dict(ctx=[0, 0, 0]),
    "full": dict(ctx=[100, 33], spare=0),
    "shared": dict(ctx=[200, 180, 150, 90] * 3, groups=4, common=4),
    "sparse": dict(ctx=[513, 40, 1000], spare=5000),
    "b300": dict(ctx=[(37 * i) % 900 + 64 for i in range(300)], groups=5, common=4, spare=1500),
    "large_pool": dict(ctx=[4171, 513] * 8, spare=299000),
    "b8192": dict(ctx=[i % 50 for i in range(8192)], spare=777),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", list(COMPACTIONS))
def test_compact(case, in_place):
    s = State(**COMPACTIONS[case])
    used = s.cursor
    _, bad = _compact(s, used, in_place, free_more=5 if in_place else 0)
    assert bad is None


def test_compact_the_largest_pool():
    s = State([40, 7168, 3], spare=2**20 - 452)
    assert s.num_blocks == 2**20
    assert _compact(s, 452, False)[1] is None


@pytest.mark.parametrize("in_place", [False, True])
def test_compactions_with_errors(in_place):
    s = State([100, 90, 64], spare=400)
    moves = ref.compact(s.ctx, s.tables, s.shares, s.free, s.cursor, s.num_blocks, 1000)[6][1]
    assert _compact(s, int(moves) - 1, in_place) == (moves, ("moves", moves))
    for c in (-1, 16 * s.tables.shape[1] + 1):
        s = State([100, 90, 64], spare=400)
        s.ctx[1] = c
        assert _compact(s, 50, in_place) == (1, ("request", 1))
    for page in (-1, 10**7):
        s = State([100, 90, 64], spare=400)
        s.tables[1, 2] = page
        assert _compact(s, 50, in_place) == (1, ("request", 1))


# ----------------------------------------------------------------- together --

def test_a_captured_round_of_forks_and_releases_advances_itself():
    """Fork two children, give them tokens, release them: ten replays equal ten
    rounds of the loops."""
    s = State([100, 33, 0, 0], cols=9, spare=30)
    d = s.device(True)
    st = torch.cuda.Stream()
    new, total = i32([0, 0, 20, 3]), 23
    more = dict(slot_mapping=torch.zeros(total, dtype=torch.int64, device="cuda"), positions=i32([0] * total),
                query_start_loc=i32([0] * 5))
    src, dst = i32([0, 0]), i32([0, 0])
    keep = i32([100, 33, 0, 0])
    pa.init()
    st.wait_stream(torch.cuda.current_stream())
    lens = d["context_lens"]
    calls = [
        pa.prepare_fork_requests(i32([0, 1]), i32([2, 3]), None, lens, d["block_tables"], d["shares_in"], d["shares_in"],
                                 d["free_pages"], d["cursor_in"], d["cursor_in"], lens, src, dst, stream=st),
        pa.prepare_build_step_metadata(lens, new, d["block_tables"], d["free_pages"], s.num_blocks, more["slot_mapping"],
                                       more["positions"], lens, more["query_start_loc"], d["cursor_in"], d["cursor_in"], st),
        pa.prepare_release_pages(lens, keep, d["block_tables"], d["shares_in"], d["shares_in"], d["free_pages"],
                                 d["cursor_in"], d["cursor_in"], lens, stream=st)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        for call in calls:
            call()
    from tests import step_reference as step
    for _ in range(10):
        g.replay()
        torch.cuda.synchronize()
        t, sh, ctx, cur, wsrc, wdst, bad = ref.fork([0, 1], [2, 3], None, s.ctx, s.tables, s.shares, s.free, s.cursor,
                                                    s.num_blocks)
        assert bad is None
        w = step.step_metadata(ctx.tolist(), new.tolist(), t, s.free, cur, s.num_blocks, total)
        assert np.array_equal(more["slot_mapping"].cpu().numpy(), w[1])
        s.tables = w[0]
        s.shares, s.free, out, s.cursor, bad = ref.release(w[3].tolist(), keep.tolist(), w[0], sh, s.free, w[5], s.num_blocks)
        s.ctx = out.tolist()
        assert bad is None
        _same(d, block_tables=s.tables, shares_in=s.shares, free_pages=s.free, cursor_in=[s.cursor], context_lens=s.ctx)
        assert src.tolist() == wsrc.tolist() and dst.tolist() == wdst.tolist()
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_fork_write_release_compact_attend():
    """Children attend like their parent did at the fork, whatever the parent
    writes afterwards; a release and a compaction with its copies change no bit."""
    hq, hkv, dh, layers = 8, 2, 128, 2
    s = State([100, 75, 0, 0, 0], spare=60, cols=12)
    g = torch.Generator(device="cuda").manual_seed(5)
    pools = torch.randn(layers, s.num_blocks, 2, 16, hkv, dh, generator=g, device="cuda").to(torch.bfloat16)
    caches = [(p[:, 0], p[:, 1]) for p in pools]
    d = s.device(True)
    lens, tables, shares, cursor = d["context_lens"], d["block_tables"], d["shares_in"], d["cursor_in"]
    qsl = i32(range(6))
    q = torch.randn(1, hq, dh, generator=g, device="cuda").to(torch.bfloat16).expand(5, hq, dh).contiguous()

    def attend(layer):
        used = torch.where(lens > 0, lens, torch.ones_like(lens))  # an empty request reads its first page
        t = torch.where(lens[:, None] > 0, tables, torch.zeros_like(tables))
        out, lse = pa.paged_attention(q, *caches[layer], t, used, qsl, dh ** -0.5, 1, 192)
        return torch.cat([out.flatten(1).float(), lse], 1)

    before = [attend(i) for i in range(layers)]
    src, dst = i32([0] * 3), i32([0] * 3)
    pa.fork_requests(i32([0, 0, 1]), i32([2, 3, 4]), None, lens, tables, shares, shares, d["free_pages"], cursor, cursor,
                     lens, src, dst)
    pa.copy_pages(caches, src, dst)
    assert lens.tolist() == [100, 75, 100, 100, 75]
    # the parents take new tokens: their partial pages change, their children's do not
    slots, pos = torch.zeros(14, dtype=torch.int64, device="cuda"), i32([0] * 14)
    start = i32([0] * 6)
    pa.build_step_metadata(lens, i32([9, 5, 0, 0, 0]), tables, d["free_pages"], s.num_blocks, slots, pos, lens, start, cursor,
                           cursor)
    for k, v in caches:
        pa.reshape_and_cache(torch.ones(14, hkv, dh, device="cuda", dtype=torch.bfloat16),
                             torch.ones(14, hkv, dh, device="cuda", dtype=torch.bfloat16), k, v, slots)
    assert pa.check_errors() == (pa.PA_OK, -1)
    forked = [attend(i) for i in range(layers)]
    for a, b in zip(before, forked):
        assert torch.equal(b[2], a[0]) and torch.equal(b[3], a[0]) and torch.equal(b[4], a[1])
        assert not torch.equal(b[0], a[0])
    # request 0 and one child end; the pool is compacted
    pa.release_pages(lens, i32([0, -1, 0, -1, -1]), tables, shares, shares, d["free_pages"], cursor, cursor, lens)
    moves, counts = s.num_blocks, i32([0, 0])
    src, dst = i32([0] * moves), i32([0] * moves)
    pa.compact_pages(lens, tables, tables, shares, shares, d["free_pages"], cursor, cursor, src, dst, counts)
    pa.copy_pages(caches, src, dst)
    assert pa.check_errors() == (pa.PA_OK, -1)
    n = int(counts[0])
    held = {int(p) for b in (1, 3, 4) for p in tables[b, :ref.pages(int(lens[b]))].tolist()}
    assert held == set(range(n)) and int(cursor) == n
    assert sorted(d["free_pages"][n:].tolist()) == list(range(n, s.num_blocks))
    after = [attend(i) for i in range(layers)]
    for a, b in zip(forked, after):
        for r in (1, 3, 4):
            assert torch.equal(a[r], b[r])
