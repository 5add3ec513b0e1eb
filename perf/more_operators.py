"""Cases of the operators that move a paged KV cache's pages between requests
(copy, fork, release, compaction) and of attention over it whose scores are
capped, biased by distance or masked.

`run` computes a case in plain torch operations, or, where `own` is true, with
the calls of paged_kv_cache_178_gb300.  `exact` computes it in 64 bits.

A page holds 16 tokens.  `shares[p]` counts the owners of page p beyond its
first.  `free_pages` is a stack: its entries from the cursor on are free.
"""
import math
import random

import torch

own = False

PAGE = 16
POISON = 2**31 - 1  # table columns past a request's last page
DECODE_MIX = "7168,7168,4171,513"  # the lengths of the repository's decode workload


# ---------------------------------------------------------------- the cases --

def listed():
    return [
        # the partial last pages of 16 forked requests, in the pools of four layers
        dict(name="copy_forks_n16", op="copy", kind="bf16", pairs=16, layers=4, hkv=2, dh=128, spare=64),
        # a compaction's moves: 2000 pages of 8 KV heads in two layers
        dict(name="copy_moves_n2000", op="copy", kind="bf16", pairs=2000, layers=2, hkv=8, dh=128, spare=300),
        # one prompt answered in four ways
        dict(name="fork_4_ways", op="fork", lens="4171", repeat=1, ways=4, cut=0),
        # the prompts of a large batch in three ways each, forked up to 40 tokens before their end
        dict(name="fork_b64_3_ways", op="fork", lens=DECODE_MIX, repeat=16, ways=3, cut=40),
        # a speculative step of 64 requests: up to 5 rejected tokens leave each
        dict(name="release_drafts_b64", op="release", lens=DECODE_MIX, repeat=16, ways=1, common=0, done=0.0, drop=5),
        # 240 requests in groups of four that share a prompt, half of them ended
        dict(name="release_done_b240", op="release", lens="7168,4171,5130,2050", repeat=60, ways=4, common=2000, done=0.5,
             drop=8),
        # the repository's decode batch in its pool of 2048 pages
        dict(name="compact_b4", op="compact", lens=DECODE_MIX, repeat=1, blocks=2048),
        # the repository's pool of 300000 pages, a tenth of it in use
        dict(name="compact_b96_300k", op="compact", lens=DECODE_MIX, repeat=24, blocks=300000),
        # one step of the decode batch in a layer with a window, whose first tokens stay
        dict(name="attn_window_decode_b4", op="attention", lens=DECODE_MIX, repeat=1, new=1, hq=8, hkv=2, dh=128, cap=0.0,
             bias=False, window=1024, prefix=4, docs=""),
        # 16 times that batch, scores capped
        dict(name="attn_cap_decode_b64", op="attention", lens=DECODE_MIX, repeat=16, new=1, hq=8, hkv=2, dh=128, cap=50.0,
             bias=False, window=0, prefix=0, docs=""),
        # a long prompt, scores capped
        dict(name="attn_cap_prompt_q4096", op="attention", lens="4096", repeat=1, new=4096, hq=8, hkv=2, dh=128, cap=50.0,
             bias=False, window=0, prefix=0, docs=""),
        # documents packed into one context behind a common prefix, a bias by distance, wide heads
        dict(name="attn_docs_bias_dh256", op="attention", lens="8192", repeat=1, new=8192, hq=16, hkv=2, dh=256, cap=0.0,
             bias=True, window=0, prefix=100, docs="700,2900,90,1601"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["copy", "fork", "release", "compact", "attention", "attention", "attention"])
    if op == "copy":
        dh, hkv, layers = rng.choice([128, 128, 256, 512]), rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 8)
        return dict(op=op, kind=rng.choice(["bf16", "bf16", "quant"]),
                    pairs=_spread(rng, 1, max(2, 2000 * 2048 // (dh * hkv * layers))), layers=layers, hkv=hkv, dh=dh,
                    spare=rng.randint(0, 300))
    n = rng.randint(1, 6)
    lens = ",".join(str(_spread(rng, 1, 7168)) for _ in range(n))
    if op == "fork":
        return dict(op=op, lens=lens, repeat=_spread(rng, 1, 10), ways=rng.randint(1, 5), cut=rng.choice([0, rng.randint(1, 99)]))
    if op == "release":
        return dict(op=op, lens=lens, repeat=_spread(rng, 1, 40), ways=rng.choice([1, n]), common=rng.randint(0, 1000),
                    done=rng.choice([0.0, 1.0, rng.random()]), drop=rng.randint(0, 40))
    if op == "compact":
        repeat = _spread(rng, 1, 16)
        used = sum(_pages(int(x)) for x in lens.split(",")) * repeat
        return dict(op=op, lens=lens, repeat=repeat, blocks=used + _spread(rng, 1, 300000))
    dh = rng.choice([128, 128, 256, 512])
    hkv = rng.choice([1, 2, 4]) * 128 // dh or 1
    group = rng.choice([1, 2, 4, 7, 8])
    new = rng.choice([1, 1, 1, rng.randint(2, 8), _spread(rng, 9, 1024), _spread(rng, 9, 1024)])
    n = rng.randint(1, 4)
    top = 7168 if new <= 8 else 8192 // n
    lens = [max(new, _spread(rng, 1, top)) for _ in range(n)]
    return dict(op=op, lens=",".join(map(str, lens)), repeat=1 if new > 8 else _spread(rng, 1, 16), new=new,
                hq=hkv * group, hkv=hkv, dh=dh, cap=rng.choice([0.0, 30.0, 50.0]), bias=rng.random() < 0.4,
                window=rng.choice([0, 0, _spread(rng, 1, 4096)]), prefix=rng.choice([0, 0, _spread(rng, 1, 500)]),
                docs=rng.choice(["", "", ",".join(str(_spread(rng, 1, 2000)) for _ in range(3))]))


def _ints(text, repeat):
    return [int(x) for x in text.split(",")] * repeat


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _page_bytes(case):
    """K and V of one page in one layer."""
    return 2 * case["hkv"] * case["dh"] * (9 if case["kind"] == "quant" else 2 * PAGE)


def _firsts(case, n):
    """The first keys of the documents that a request's last `new` of n tokens lie in, or None."""
    if not case["docs"]:
        return None
    sizes, starts, at = _ints(case["docs"], 1), [], 0
    while at < n:
        starts += [at] * sizes[0]
        at, sizes = at + sizes[0], sizes[1:] + sizes[:1]
    return starts[n - case["new"]:n]


def work(case):
    """Bytes that have to be read and written once, and the arithmetic."""
    if case["op"] == "copy":
        return {"bytes": case["pairs"] * (2 * case["layers"] * _page_bytes(case) + 8), "flops": 0}
    lens = _ints(case["lens"], case["repeat"])
    if case["op"] == "fork":
        n = len(lens) * case["ways"]
        pages = sum(_pages(x) for x in lens) * case["ways"]
        return {"bytes": 4 * (4 * pages + 2 * 4 * n + 2 * len(lens) + 2 * n), "flops": pages}
    if case["op"] == "release":
        gone = sum(case["done"] * (_pages(x) - case["common"] // PAGE) + (1 - case["done"]) * case["drop"] / 32 for x in lens)
        gone = int(max(1, gone))
        return {"bytes": 4 * (4 * gone + 3 * len(lens)), "flops": gone}
    if case["op"] == "compact":
        used = sum(_pages(x) for x in lens)
        return {"bytes": 4 * (2 * used + 2 * used + case["blocks"] - used + len(lens)), "flops": used}
    hq, hkv, dh, new = case["hq"], case["hkv"], case["dh"], case["new"]
    window = case["window"] or 2**31
    pairs = keys = 0
    for n in lens:
        first, prefix = _firsts(case, n) or [0] * new, min(case["prefix"], n)
        low = n
        for i in range(new):
            p = n - new + i
            lo = max(first[i], p - window + 1)
            pairs += p - lo + 1 + min(prefix, lo) + max(0, prefix - p - 1)
            low = min(low, lo)
        keys += n - low + min(prefix, low)
    return {"bytes": keys * hkv * dh * 4 + len(lens) * new * hq * (dh * 4 + 4) + 4 * (keys // PAGE + 1) + 8 * len(lens),
            "flops": 4 * pairs * hq * dh}


# --------------------------------------------------------------- the inputs --

def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _tables(counts, num_blocks, columns, g, dev):
    """A shuffled block table [B, columns] whose rows own disjoint pages, and the order of all pages."""
    counts = torch.tensor(counts, device=dev)
    start = torch.cumsum(counts, 0) - counts
    perm = torch.randperm(num_blocks, generator=g, device=dev)
    col = torch.arange(columns, device=dev)
    index = (start[:, None] + col).clamp(max=num_blocks - 1)
    return torch.where(col < counts[:, None], perm[index], POISON).to(torch.int32), perm


def prepare(case, seed):
    dev = _device()
    g = _generator(seed, dev)
    rng = random.Random(int(seed))
    s = {"op": case["op"], "case": case}
    {"copy": _prepare_copy, "fork": _prepare_fork, "release": _prepare_release, "compact": _prepare_compact,
     "attention": _prepare_attention}[case["op"]](s, case, dev, g, rng)
    if own:
        s["calls"] = _calls(s)
    return s


def _prepare_copy(s, case, dev, g, rng):
    n, hkv, dh = case["pairs"], case["hkv"], case["dh"]
    blocks = 2 * n + case["spare"]
    if case["kind"] == "quant":
        s["pools"] = torch.randint(0, 256, (case["layers"], blocks, 2, hkv, 9 * dh), generator=g, device=dev, dtype=torch.uint8)
    else:
        s["pools"] = torch.randn(case["layers"], blocks, 2, PAGE, hkv, dh, generator=g, device=dev, dtype=torch.bfloat16)
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    s["src_pages"], s["dst_pages"] = order[:n].contiguous(), order[n:2 * n].contiguous()


def _prepare_fork(s, case, dev, g, rng):
    # every parent's context is some tokens off the listed length, from the seed
    longest = _ints(case["lens"], case["repeat"])
    parents = [max(1, n - rng.randint(0, 40)) for n in longest]
    n = len(parents) * case["ways"]
    forks = [max(0, p - rng.randint(0, case["cut"])) for p in parents for _ in range(case["ways"])]
    ctx = parents + [0] * n
    used = sum(_pages(x) for x in parents)
    blocks = sum(_pages(x) for x in longest) + n + 40
    tables, perm = _tables([_pages(x) for x in ctx], blocks, max(_pages(x) for x in longest) + 2, g, dev)
    shares = torch.zeros(blocks, dtype=torch.int32, device=dev)
    shares[perm[:used]] = torch.randint(0, 3, (used,), generator=g, device=dev, dtype=torch.int32)
    s.update(parents=_i32([i for i in range(len(parents)) for _ in range(case["ways"])], dev),
             children=_i32([len(parents) + i for i in range(n)], dev), fork_lens=_i32(forks, dev), context_lens=_i32(ctx, dev),
             block_tables=tables, shares_in=shares, shares_out=torch.zeros_like(shares), num_blocks=blocks,
             free_pages=perm[used - 3 if used > 3 else used:].to(torch.int32).contiguous(),
             cursor_in=_i32([3 if used > 3 else 0], dev), cursor_out=_i32([-1], dev),
             seq_lens=torch.zeros(len(ctx), dtype=torch.int32, device=dev),
             copy_src=torch.zeros(n, dtype=torch.int32, device=dev), copy_dst=torch.zeros(n, dtype=torch.int32, device=dev))


def _prepare_release(s, case, dev, g, rng):
    # groups of `ways` requests share the pages of their first `common` tokens
    ways, common = case["ways"], case["common"] // PAGE
    if ways == 1:
        common = 0
    longest = [common * PAGE + max(1, n - case["common"]) for n in _ints(case["lens"], case["repeat"])]
    ctx = [max(common * PAGE + 1, n - rng.randint(0, 40)) for n in longest]
    keep = [0 if rng.random() < case["done"] else max(common * PAGE, n - rng.randint(0, case["drop"])) for n in ctx]
    groups = [i // ways for i in range(len(ctx))]
    private = [_pages(n) - common for n in ctx]
    used = sum(private) + common * (groups[-1] + 1)
    blocks = sum(_pages(n) - common for n in longest) + common * (groups[-1] + 1) + 50
    columns = max(_pages(n) for n in longest) + 1
    rows, perm = _tables(private, blocks, columns, g, dev)
    tables = torch.full((len(ctx), columns), POISON, dtype=torch.int32, device=dev)
    tables[:, common:] = rows[:, :columns - common]
    heads = perm[sum(private):used].view(groups[-1] + 1, common)
    tables[:, :common] = heads[torch.tensor(groups, device=dev)].to(torch.int32)
    shares = torch.zeros(blocks, dtype=torch.int32, device=dev)
    sizes = torch.bincount(torch.tensor(groups, device=dev)) - 1
    shares[heads.flatten()] = sizes.repeat_interleave(common).to(torch.int32)
    free = torch.full((blocks,), -5, dtype=torch.int32, device=dev)
    free[used:] = perm[used:].to(torch.int32)
    s.update(context_lens=_i32(ctx, dev), keep_lens=_i32(keep, dev), block_tables=tables, shares_in=shares,
             shares_out=torch.zeros_like(shares), num_blocks=blocks, free_pages=free, cursor_in=_i32([used], dev),
             cursor_out=_i32([-1], dev), seq_lens=torch.zeros(len(ctx), dtype=torch.int32, device=dev))


def _prepare_compact(s, case, dev, g, rng):
    longest = _ints(case["lens"], case["repeat"])
    counts = [_pages(max(0, n - rng.randint(0, 40))) for n in longest]
    ctx = [max(0, n * PAGE - rng.randint(0, 15)) for n in counts]
    used, blocks, most = sum(counts), case["blocks"], sum(_pages(n) for n in longest)
    tables, perm = _tables(counts, blocks, max(_pages(n) for n in longest) + 1, g, dev)
    shares = torch.zeros(blocks, dtype=torch.int32, device=dev)
    shares[perm[:used]] = torch.randint(0, 3, (used,), generator=g, device=dev, dtype=torch.int32)
    free = torch.full((blocks,), -5, dtype=torch.int32, device=dev)
    free[used:] = perm[used:].to(torch.int32)
    s.update(context_lens=_i32(ctx, dev), block_tables=tables, tables_out=tables.clone(), shares_in=shares,
             shares_out=torch.zeros_like(shares), num_blocks=blocks, free_pages=free, cursor_in=_i32([used], dev),
             cursor_out=_i32([-1], dev), copy_src=torch.zeros(most, dtype=torch.int32, device=dev),
             copy_dst=torch.zeros(most, dtype=torch.int32, device=dev),
             counts=torch.zeros(2, dtype=torch.int32, device=dev))


def _prepare_attention(s, case, dev, g, rng):
    lens, hq, hkv, dh, new = _ints(case["lens"], case["repeat"]), case["hq"], case["hkv"], case["dh"], case["new"]
    total = sum(_pages(n) for n in lens)
    blocks = total + 8
    tables, _ = _tables([_pages(n) for n in lens], blocks, max(_pages(n) for n in lens) + 1, g, dev)
    pool = torch.randn(blocks, 2, PAGE, hkv, dh, generator=g, device=dev, dtype=torch.bfloat16)
    tokens = len(lens) * new
    # wide scores, so that a cap has something to do
    q = torch.randn(tokens, hq, dh, generator=g, device=dev) * (4.0 if case["cap"] else 1.0)
    s.update(k_cache=pool[:, 0], v_cache=pool[:, 1], block_tables=tables, seq_lens=_i32(lens, dev), q=q.to(torch.bfloat16),
             query_start_loc=torch.arange(len(lens) + 1, dtype=torch.int32, device=dev) * new, scale=1.0 / math.sqrt(dh),
             max_query_len=new, max_seq_len=max(lens), slopes=None, prefix_lens=None, first_keys=None,
             out=torch.zeros(tokens, hq, dh, dtype=torch.bfloat16, device=dev),
             lse=torch.zeros(tokens, hq, dtype=torch.float32, device=dev))
    if case["bias"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, dtype=torch.float32, device=dev) / hq)
    if case["prefix"]:
        s["prefix_lens"] = _i32([min(case["prefix"], n) for n in lens], dev)
    if case["docs"]:
        s["first_keys"] = _i32([x for n in lens for x in _firsts(case, n)], dev)


def _calls(s):
    """The handles that a program keeps: calls validated once, their workspace."""
    from paged_kv_cache_178_gb300 import pagedattn as pa
    if s["op"] == "copy":
        if s["case"]["kind"] == "quant":
            pools = [pa.QuantCache(p[:, 0], p[:, 1], s["case"]["dh"]) for p in s["pools"]]
            return [pa.prepare_copy_pages_quant(pools, s["src_pages"], s["dst_pages"])]
        return [pa.prepare_copy_pages([(p[:, 0], p[:, 1]) for p in s["pools"]], s["src_pages"], s["dst_pages"])]
    if s["op"] == "fork":
        return [pa.prepare_fork_requests(
            s["parents"], s["children"], s["fork_lens"], s["context_lens"], s["block_tables"], s["shares_in"], s["shares_out"],
            s["free_pages"], s["cursor_in"], s["cursor_out"], s["seq_lens"], s["copy_src"], s["copy_dst"])]
    if s["op"] == "release":
        return [pa.prepare_release_pages(
            s["context_lens"], s["keep_lens"], s["block_tables"], s["shares_in"], s["shares_out"], s["free_pages"],
            s["cursor_in"], s["cursor_out"], s["seq_lens"])]
    if s["op"] == "compact":
        return [pa.prepare_compact_pages(
            s["context_lens"], s["block_tables"], s["tables_out"], s["shares_in"], s["shares_out"], s["free_pages"],
            s["cursor_in"], s["cursor_out"], s["copy_src"], s["copy_dst"], s["counts"],
            pa.new_compact_workspace(s["num_blocks"], device=s["context_lens"].device))]
    case, bounds = s["case"], (s["max_query_len"], s["max_seq_len"])
    ws = pa.new_scored_workspace(s["seq_lens"].numel(), case["hq"], case["hkv"], case["dh"], *bounds, device=s["q"].device)
    return [pa.prepare_paged_attention_scored(
        s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["seq_lens"], s["query_start_loc"], s["scale"], *bounds,
        s["out"], s["lse"], ws, soft_cap=case["cap"], slopes=s["slopes"], window=case["window"], prefix_lens=s["prefix_lens"],
        first_keys=s["first_keys"])]


_OUTPUTS = {
    "copy": ["pools"],
    "fork": ["block_tables", "shares_out", "seq_lens", "cursor_out", "copy_src", "copy_dst"],
    "release": ["shares_out", "free_pages", "cursor_out", "seq_lens"],
    "compact": ["tables_out", "shares_out", "free_pages", "cursor_out", "copy_src", "copy_dst", "counts"],
    "attention": ["out", "lse"],
}


def run(s):
    if own:
        for call in s["calls"]:
            call()
        return [s[name] for name in _OUTPUTS[s["op"]]]
    return {"copy": _plain_copy, "fork": _plain_fork, "release": _plain_release, "compact": _plain_compact,
            "attention": _plain_attention}[s["op"]](s)


# ---------------------------------------------------------- the plain forms --

def _plain_copy(s):
    s["pools"][:, s["dst_pages"].long()] = s["pools"][:, s["src_pages"].long()]
    return [s["pools"]]


def _exclusive(counts):
    return torch.cumsum(counts, 0) - counts


def _plain_fork(s):
    """Whole pages of the parent are shared, a partial one gets a page of its own."""
    parents, children, lens = s["parents"].long(), s["children"].long(), s["fork_lens"].long()
    full, tail = lens // PAGE, lens % PAGE > 0
    fresh = s["free_pages"].long()[(s["cursor_in"].long() + _exclusive(tail.long())).clamp(max=s["free_pages"].numel() - 1)]
    tables = s["block_tables"]
    rows = tables[parents].long()
    col = torch.arange(tables.shape[1], device=lens.device)
    shared = col < full[:, None]
    shares = s["shares_in"].long()
    ids = torch.where(shared, rows, 0)
    shares = shares.index_add(0, ids.flatten(), shared.long().flatten())
    source = torch.gather(rows, 1, full[:, None]).squeeze(1)
    new = torch.where(shared, rows, tables[children].long())
    new = torch.where((col == full[:, None]) & tail[:, None], fresh[:, None], new)
    tables[children] = new.to(torch.int32)
    seq_lens = s["context_lens"].clone()
    seq_lens[children] = lens.to(torch.int32)
    return [tables, shares.to(torch.int32), seq_lens, (s["cursor_in"] + tail.sum()).to(torch.int32),
            torch.where(tail, source, -1).to(torch.int32), torch.where(tail, fresh, -1).to(torch.int32)]


def _plain_release(s):
    """Pages past the kept tokens lose an owner; those without one go onto the free stack."""
    ctx, keep = s["context_lens"].long(), s["keep_lens"].long()
    col = torch.arange(s["block_tables"].shape[1], device=ctx.device)
    gone = (col >= ((keep + PAGE - 1) // PAGE)[:, None]) & (col < ((ctx + PAGE - 1) // PAGE)[:, None])
    ids = s["block_tables"].long()[gone]  # in order of request and column
    at = torch.arange(ids.numel(), device=ctx.device)
    shares = s["shares_in"].long().index_add(0, ids, -torch.ones_like(ids))
    last = torch.full_like(shares, -1).scatter_reduce(0, ids, at, "amax")
    freed = ids[(shares[ids] < 0) & (last[ids] == at)]
    cursor = s["cursor_in"].long() - freed.numel()
    free = s["free_pages"]
    free[cursor + torch.arange(freed.numel(), device=ctx.device)] = freed.to(torch.int32)
    return [shares.clamp(min=0).to(torch.int32), free, cursor.to(torch.int32), s["keep_lens"].clone()]


def _plain_compact(s):
    """The k-th page in use from n on moves to the k-th unused one below n."""
    tables, blocks = s["block_tables"].long(), s["num_blocks"]
    col = torch.arange(tables.shape[1], device=tables.device)
    used = col < ((s["context_lens"].long() + PAGE - 1) // PAGE)[:, None]
    live = torch.zeros(blocks, dtype=torch.bool, device=tables.device)
    live[tables[used]] = True
    n = live.sum()
    page = torch.arange(blocks, device=tables.device)
    src, dst = page[live & (page >= n)], page[~live & (page < n)]
    place = page.clone()
    place[src] = dst
    moved = torch.where(used, place[torch.where(used, tables, 0)], s["tables_out"].long())
    shares = torch.zeros_like(s["shares_in"])
    shares[place[live]] = s["shares_in"][live]
    free = s["free_pages"].long()
    at = page - (free.numel() - blocks)
    free = torch.where(at >= n, at, free)
    fill = torch.full_like(s["copy_src"], -1)
    copy_src, copy_dst = fill.clone(), fill
    copy_src[:src.numel()] = src.to(torch.int32)
    copy_dst[:dst.numel()] = dst.to(torch.int32)
    s["free_pages"].copy_(free)
    return [moved.to(torch.int32), shares, s["free_pages"], (free.numel() - blocks + n).to(torch.int32).reshape(1), copy_src,
            copy_dst, torch.stack([n, (live & (page >= n)).sum()]).to(torch.int32)]


def _seen(s, keys):
    """Which of `keys` key positions each new token sees, and its distance to them, [B, new, keys]."""
    lens, new = s["seq_lens"].long(), s["case"]["new"]
    key = torch.arange(keys, device=lens.device)
    dist = (lens[:, None] - new + torch.arange(new, device=lens.device))[..., None] - key
    seen = dist >= 0
    if s["case"]["window"]:
        seen &= dist < s["case"]["window"]
    if s["first_keys"] is not None:
        seen &= key >= s["first_keys"].view(-1, new, 1)
    if s["prefix_lens"] is not None:
        seen |= key < s["prefix_lens"].view(-1, 1, 1)
    return seen & (key < lens.view(-1, 1, 1)), dist.abs()


def _plain_attention(s):
    """Softmax attention over the padded contexts."""
    case, lens = s["case"], s["seq_lens"].long()
    hq, hkv, dh, new = case["hq"], case["hkv"], case["dh"], case["new"]
    batch, group, columns = lens.numel(), hq // hkv, _pages(s["max_seq_len"])
    col = torch.arange(columns, device=lens.device)
    have = col < ((lens + PAGE - 1) // PAGE)[:, None]
    ids = torch.where(have, s["block_tables"][:, :columns].long(), 0)
    k, v = (c[ids].flatten(1, 2).float().permute(0, 2, 1, 3) for c in (s["k_cache"], s["v_cache"]))
    q = s["q"].float().view(batch, new, hkv, group, dh).permute(0, 2, 3, 1, 4).flatten(2, 3)
    z = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).unflatten(2, (group, new))
    if case["cap"]:
        z = case["cap"] * torch.tanh(z / case["cap"])
    seen, dist = _seen(s, columns * PAGE)
    if s["slopes"] is not None:
        z = z - s["slopes"].view(1, hkv, group, 1, 1) * dist[:, None, None].float()
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e38)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (group, new)) / total.clamp(min=1e-38)
    lse = (top + torch.log(total)).squeeze(-1)
    return [out.permute(0, 3, 1, 2, 4).reshape(batch * new, hq, dh).to(torch.bfloat16),
            lse.permute(0, 3, 1, 2).reshape(batch * new, hq)]


# ----------------------------------------------------------- in 64 bits -----

def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(prepare(case, seed))
    if case["op"] == "copy" and case["kind"] == "bf16":
        s = prepare(case, seed)
        pools = s["pools"].double()
        for i, j in zip(s["src_pages"].tolist(), s["dst_pages"].tolist()):
            pools[:, j] = pools[:, i]
        return [pools]
    return None  # whole numbers


def _exact_attention(s):
    case = s["case"]
    hq, group, new = case["hq"], case["hq"] // case["hkv"], case["new"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
    first = None if s["first_keys"] is None else s["first_keys"].long()
    for b, n in enumerate(s["seq_lens"].tolist()):
        ids = s["block_tables"][b, :_pages(n)].long()
        rows = slice(b * new, (b + 1) * new)
        j = torch.arange(n, device=ids.device)
        p = torch.arange(n - new, n, device=ids.device).unsqueeze(1)
        low = torch.zeros_like(p) if first is None else first[rows].unsqueeze(1)
        if case["window"]:
            low = torch.maximum(low, p - case["window"] + 1)
        hidden = (j > p) | (j < low)
        if s["prefix_lens"] is not None:
            hidden &= j >= s["prefix_lens"][b]
        for h in range(hq):
            k, v = (c[ids, :, h // group].reshape(-1, case["dh"])[:n].double() for c in (s["k_cache"], s["v_cache"]))
            t = s["q"][rows, h].double() @ k.T * s["scale"]
            if case["cap"]:
                e = torch.expm1(2 * t / case["cap"])
                t = case["cap"] * torch.where(torch.isinf(e), torch.ones_like(e), e / (e + 2))
            if s["slopes"] is not None:
                t -= s["slopes"][h].double() * (p - j).abs()
            t[hidden] = -math.inf
            lse[rows, h] = torch.logsumexp(t, 1)
            out[rows, h] = torch.exp(t - lse[rows, h, None]) @ v
    return [out, lse]
