"""Operator cases around the paged KV cache: the metadata of a serving step
built on the GPU, the per-head norm and position rotation of queries and keys,
the write and read-back of a cache held in 4 bits, and attention over it.

`run` computes a case in plain torch operations, or, where `own` is true, with
the calls of paged_kv_cache_178_gb300.  `exact` computes it in 64 bits.

The 4-bit cache: a page holds 16 tokens; for one page and KV head the K record
is [16 tokens][Dh/2 bytes] of codes, then [16 tokens][Dh/16] scales; the V
record is [Dh/2][16 tokens] of codes, then [Dh/16][16 tokens] scales.  A byte
holds the e2m1 codes of two neighbouring head-dim elements (the even one in the
low half); a scale byte is the e4m3 factor of 16 neighbouring elements.
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
        # a decode step of 64 requests: one new token each
        dict(name="metadata_decode_b64", op="metadata", ctx=DECODE_MIX, new="1,1,1,1", repeat=16, pad=0),
        # a mixed step: chunks of prompts beside decodes and idle requests, padded to a fixed token count
        dict(name="metadata_mixed_b240", op="metadata", ctx="0,513,1000,4171,7168,0,31,16", new="1024,1,0,257,1,700,64,1",
             repeat=30, pad=640),
        # one layer's decode step of 64 requests: norm, rotation and the cache write
        dict(name="rope_decode_t64", op="rope", tokens=64, hq=8, hkv=2, dh=128, rot=128, interleaved=False, cache=True,
             norm=True, far=8192),
        # a prompt batch of a model with 32 query heads
        dict(name="rope_prompt_t16384", op="rope", tokens=16384, hq=32, hkv=8, dh=128, rot=128, interleaved=False,
             cache=True, norm=True, far=65536),
        # wide heads, a quarter of each rotated, neighbouring pairs, no cache write, an odd count
        dict(name="rope_partial_dh256", op="rope", tokens=4099, hq=16, hkv=2, dh=256, rot=64, interleaved=True,
             cache=False, norm=True, far=32768),
        # a chunk of four prompts goes into the 4-bit cache and their whole contexts are read back
        dict(name="quant_chunk_b4", op="quant", lens=DECODE_MIX, repeat=1, new=128, hkv=2, dh=128),
        # the same for a large batch and 8 KV heads
        dict(name="quant_large_b16", op="quant", lens="4096,4003,7168,1117", repeat=4, new=1024, hkv=8, dh=128),
        # the repository's decode batch, and 16 times it
        dict(name="attn_decode_b4", op="attention", lens=DECODE_MIX, repeat=1, new=1, hq=8, hkv=2, dh=128),
        dict(name="attn_decode_b64", op="attention", lens=DECODE_MIX, repeat=16, new=1, hq=8, hkv=2, dh=128),
        # a long document beside two short ones, eight query heads to a KV head
        dict(name="attn_decode_long", op="attention", lens="131072,9001,700", repeat=1, new=1, hq=32, hkv=4, dh=128),
        # five drafted tokens a request, wide heads
        dict(name="attn_draft_dh256", op="attention", lens="4171,2050,977,5000", repeat=4, new=5, hq=8, hkv=2, dh=256),
        # a chunk of two long prompts
        dict(name="attn_chunk_q1024", op="attention", lens="9216,5130", repeat=1, new=1024, hq=8, hkv=2, dh=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["metadata", "rope", "quant", "attention", "attention"])
    if op == "metadata":
        n = rng.randint(1, 8)
        return dict(op=op, ctx=",".join(str(rng.choice([0, _spread(rng, 1, 8000)])) for _ in range(n)),
                    new=",".join(str(rng.choice([0, 1, 1, _spread(rng, 1, 1000)])) for _ in range(n)),
                    repeat=_spread(rng, 1, 240 // n), pad=rng.choice([0, rng.randint(1, 500)]))
    if op == "rope":
        dh = rng.choice([128, 128, 256, 512])
        hkv = rng.choice([1, 2, 4, 8]) * 128 // dh or 1
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        return dict(op=op, tokens=min(_spread(rng, 1, 16384), 16384 * 48 * 128 // ((hq + 2 * hkv) * dh)), hq=hq, hkv=hkv,
                    dh=dh, rot=rng.choice([dh, dh, dh // 2, 64]), interleaved=rng.random() < 0.3,
                    cache=rng.random() < 0.6, norm=rng.random() < 0.8, far=_spread(rng, 64, 65536))
    dh = rng.choice([128, 128, 256, 512])
    n = rng.randint(1, 4)
    if op == "quant":
        hkv = rng.choice([1, 2, 4, 8])
        top = 4096 * 128 // dh
        lens = [_spread(rng, 1, top) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), repeat=rng.randint(1, 4), new=rng.choice([1, _spread(rng, 1, 1024)]),
                    hkv=hkv, dh=dh)
    hkv = rng.choice([1, 2, 4]) * 128 // dh or 1
    group = rng.choice([1, 2, 4, 7, 8])
    new = rng.choice([1, 1, 1, 2, rng.randint(3, 8), _spread(rng, 9, 512)])
    lens = [max(new, _spread(rng, 1, 7168)) for _ in range(n)]
    return dict(op=op, lens=",".join(map(str, lens)), repeat=rng.choice([1, 1, 2]) if new > 8 else _spread(rng, 1, 16),
                new=new, hq=hkv * group, hkv=hkv, dh=dh)


def _ints(text, repeat):
    return [int(x) for x in text.split(",")] * repeat


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    """Bytes that have to be read and written once, and the arithmetic."""
    if case["op"] == "metadata":
        ctx, new = _ints(case["ctx"], case["repeat"]), _ints(case["new"], case["repeat"])
        b, t = len(ctx), sum(new) + case["pad"]
        table = sum(_pages(c + n) - _pages(c) for c, n in zip(ctx, new))
        read_pages = sum(_pages(c + n) - c // PAGE for c, n in zip(ctx, new) if n)
        return {"bytes": 4 * (2 * b + read_pages + table + 2 * b + 1 + 2) + 12 * t, "flops": 4 * b + 4 * t}
    if case["op"] == "rope":
        t, dh = case["tokens"], case["dh"]
        heads = case["hq"] + case["hkv"] * (2 if case["cache"] else 1)
        return {"bytes": t * (heads * dh * 4 + 4 * case["rot"] + 4 + (8 if case["cache"] else 0)),
                "flops": t * (case["hq"] + case["hkv"]) * dh * 8}
    hkv, dh = case["hkv"], case["dh"]
    lens = _ints(case["lens"], case["repeat"])
    token = hkv * dh * 2  # elements of K and V
    if case["op"] == "quant":
        new = sum(min(case["new"], n) for n in lens)
        pages = sum(_pages(n) for n in lens)
        return {"bytes": new * (token * 2 + token * 9 // 16 + 8) + pages * PAGE * (token * 9 // 16 + token * 2) + 8 * pages,
                "flops": (new + pages * PAGE) * token * 4}
    hq, new = case["hq"], case["new"]
    pairs = sum(new * n - new * (new - 1) // 2 for n in lens)
    return {"bytes": sum(lens) * token * 9 // 16 + len(lens) * new * hq * (dh * 4 + 4) + sum(_pages(n) for n in lens) * 4,
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


def _tables(lens, num_blocks, columns, g, dev):
    """A shuffled block table [B, columns] whose rows own disjoint pages."""
    counts = torch.tensor([_pages(n) for n in lens], device=dev)
    start = torch.cumsum(counts, 0) - counts
    perm = torch.randperm(num_blocks, generator=g, device=dev)
    col = torch.arange(columns, device=dev)
    index = (start[:, None] + col).clamp(max=num_blocks - 1)
    return torch.where(col < counts[:, None], perm[index], POISON).to(torch.int32), perm


def _slots_of_last(tables, lens, new, dev):
    """The slots of each request's last min(new, length) tokens."""
    lens = torch.tensor(lens, device=dev)
    pos = lens[:, None] - new + torch.arange(new, device=dev)
    page = torch.gather(tables.long(), 1, pos.clamp(min=0) // PAGE)
    return (page * PAGE + pos.clamp(min=0) % PAGE)[pos >= 0]


def prepare(case, seed):
    dev = _device()
    g = _generator(seed, dev)
    rng = random.Random(int(seed))
    s = {"op": case["op"], "case": case}
    if case["op"] == "metadata":
        # every request's context is some tokens off the listed length, from the seed
        ctx = [max(0, c - rng.randint(0, 40)) for c in _ints(case["ctx"], case["repeat"])]
        new = _ints(case["new"], case["repeat"])
        total = sum(new) + case["pad"]
        columns = max(_pages(c + n) for c, n in zip(_ints(case["ctx"], case["repeat"]), new)) + 2
        old = sum(_pages(c) for c in ctx)
        free = sum(_pages(c + n) - _pages(c) for c, n in zip(ctx, new)) + 9
        blocks = old + free + 32
        tables, perm = _tables(ctx, blocks, columns, g, dev)
        s.update(context_lens=_i32(ctx, dev), query_lens=_i32(new, dev), block_tables=tables, num_blocks=blocks,
                 free_pages=perm[old:old + free + 5].to(torch.int32).contiguous(), cursor_in=_i32([5], dev),
                 cursor_out=_i32([-1], dev), slot_mapping=torch.full((total,), -7, dtype=torch.int64, device=dev),
                 positions=torch.full((total,), -7, dtype=torch.int32, device=dev),
                 seq_lens=torch.zeros(len(ctx), dtype=torch.int32, device=dev),
                 query_start_loc=torch.zeros(len(ctx) + 1, dtype=torch.int32, device=dev))
    elif case["op"] == "rope":
        t, hq, hkv, dh, rot = case["tokens"], case["hq"], case["hkv"], case["dh"], case["rot"]
        qkv = torch.randn(t, (hq + 2 * hkv) * dh, generator=g, device=dev).to(torch.bfloat16)
        far = case["far"]
        angle = torch.arange(far, dtype=torch.float64, device=dev)[:, None] * torch.exp(
            torch.arange(0, rot, 2, dtype=torch.float64, device=dev) * (-math.log(10000.0) / rot))
        s.update(q=qkv[:, :hq * dh].view(t, hq, dh), k=qkv[:, hq * dh:(hq + hkv) * dh].view(t, hkv, dh),
                 v=qkv[:, (hq + hkv) * dh:].view(t, hkv, dh),
                 cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float().contiguous(),
                 positions=torch.randint(0, far, (t,), generator=g, device=dev, dtype=torch.int32), eps=1e-6,
                 q_out=torch.zeros(t, hq, dh, dtype=torch.bfloat16, device=dev))
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.2 * torch.randn(dh, generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
        if case["cache"]:
            blocks = _pages(t) + 3
            s["slots"] = torch.randperm(blocks * PAGE, generator=g, device=dev)[:t]
            s["k_cache"], s["v_cache"] = torch.zeros(2, blocks, PAGE, hkv, dh, dtype=torch.bfloat16, device=dev).unbind(0)
        else:
            s["k_out"] = torch.zeros(t, hkv, dh, dtype=torch.bfloat16, device=dev)
    else:
        lens, hkv, dh = _ints(case["lens"], case["repeat"]), case["hkv"], case["dh"]
        total = sum(_pages(n) for n in lens)
        blocks, columns = total + 8, max(_pages(n) for n in lens) + 1
        tables, _ = _tables(lens, blocks, columns, g, dev)
        s.update(block_tables=tables, seq_lens=_i32(lens, dev), k_scale=0.5, v_scale=1.0, total=total)
        for name in ("k", "v"):
            # channels of different strength, as keys have them
            x = torch.randn(blocks, PAGE, hkv, dh, generator=g, device=dev)
            x = (x * torch.exp(0.3 * torch.randn(hkv, dh, generator=g, device=dev))).to(torch.bfloat16)
            codes, scales = _quantise(x, s[name + "_scale"])
            s[name + "_pool"] = _records(codes, scales, name)
            del x, codes, scales
        if case["op"] == "quant":
            s["slots"] = _slots_of_last(tables, lens, case["new"], dev)
            n = s["slots"].numel()
            kv = torch.randn(n, 2 * hkv * dh, generator=g, device=dev).to(torch.bfloat16)
            s["key"], s["value"] = kv[:, :hkv * dh].view(n, hkv, dh), kv[:, hkv * dh:].view(n, hkv, dh)
            s["k_out"], s["v_out"] = torch.zeros(2, total, PAGE, hkv, dh, dtype=torch.bfloat16, device=dev).unbind(0)
            s["compact_tables"] = torch.zeros_like(tables)
            s["compact_offsets"] = torch.zeros(len(lens) + 1, dtype=torch.int32, device=dev)
        else:
            new, hq = case["new"], case["hq"]
            s["q"] = torch.randn(len(lens) * new, hq, dh, generator=g, device=dev).to(torch.bfloat16)
            s["query_start_loc"] = torch.arange(len(lens) + 1, dtype=torch.int32, device=dev) * new
            s["scale"] = 1.0 / math.sqrt(dh)
            s["max_seq_len"], s["max_query_len"] = max(lens), new
            s["out"] = torch.zeros_like(s["q"])
            s["lse"] = torch.zeros(len(lens) * new, hq, device=dev)
    if own:
        s["calls"] = _calls(s)
    return s


def _calls(s):
    """The handles that a program keeps: calls validated once, their workspace."""
    from paged_kv_cache_178_gb300 import pagedattn as pa
    if s["op"] == "metadata":
        return [pa.prepare_build_step_metadata(
            s["context_lens"], s["query_lens"], s["block_tables"], s["free_pages"], s["num_blocks"], s["slot_mapping"],
            s["positions"], s["seq_lens"], s["query_start_loc"], s["cursor_out"], cursor_in=s["cursor_in"])]
    if s["op"] == "rope":
        extra = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], interleaved=s["case"]["interleaved"])
        if s["case"]["cache"]:
            return [pa.prepare_qk_norm_rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["q_out"],
                                                      s["k_cache"], s["v_cache"], s["slots"], **extra)]
        return [pa.prepare_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_out"], s["k_out"], **extra)]
    cache = pa.QuantCache(s["k_pool"], s["v_pool"], s["case"]["dh"], s["k_scale"], s["v_scale"])
    if s["op"] == "quant":
        return [pa.prepare_reshape_and_cache_quant(s["key"], s["value"], cache, s["slots"]),
                pa.prepare_dequantize_kv(cache, s["block_tables"], s["seq_lens"], s["k_out"], s["v_out"],
                                         s["compact_tables"], s["compact_offsets"])]
    bounds = (s["max_query_len"], s["max_seq_len"])
    ws = pa.new_quant_workspace(s["seq_lens"].numel(), s["case"]["hq"], s["case"]["hkv"], s["case"]["dh"], *bounds,
                                device=s["q"].device)
    return [pa.prepare_paged_attention_quant(s["q"], cache, s["block_tables"], s["seq_lens"], s["query_start_loc"],
                                             s["scale"], *bounds, s["out"], s["lse"], ws)]


def run(s):
    if own:
        for call in s["calls"]:
            call()
        return [s[name] for name in _outputs(s)]
    return {"metadata": _plain_metadata, "rope": _plain_rope, "quant": _plain_quant, "attention": _plain_attention}[s["op"]](s)


def _outputs(s):
    if s["op"] == "metadata":
        return ["block_tables", "slot_mapping", "positions", "seq_lens", "query_start_loc", "cursor_out"]
    if s["op"] == "rope":
        return ["q_out", "k_cache", "v_cache"] if s["case"]["cache"] else ["q_out", "k_out"]
    if s["op"] == "quant":
        return ["k_out", "v_out", "compact_tables", "compact_offsets"]
    return ["out", "lse"]


# ---------------------------------------------------------- the plain forms --

def _exclusive(counts):
    return torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])


def _plain_metadata(s):
    """New pages from the free list, then each new token's slot and position."""
    ctx, new = s["context_lens"].long(), s["query_lens"].long()
    tables, columns = s["block_tables"].long(), s["block_tables"].shape[1]
    have = (ctx + PAGE - 1) // PAGE
    need = (ctx + new + PAGE - 1) // PAGE - have
    first = _exclusive(need)
    col = torch.arange(columns, device=ctx.device)
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    take = s["cursor_in"].long() + first[:-1, None] + col - have[:, None]
    tables = torch.where(fresh, s["free_pages"].long()[take.clamp(0, s["free_pages"].numel() - 1)], tables)
    loc = _exclusive(new)
    token = torch.arange(s["slot_mapping"].numel(), device=ctx.device)
    req = (torch.searchsorted(loc, token, right=True) - 1).clamp(max=ctx.numel() - 1)
    live = token < loc[-1]
    pos = torch.where(live, ctx[req] + token - loc[req], 0)
    slot = tables[req, pos // PAGE] * PAGE + pos % PAGE
    return [tables.to(torch.int32), torch.where(live, slot, -1), torch.where(live, pos, -1).to(torch.int32),
            (ctx + new).to(torch.int32), loc.to(torch.int32), (s["cursor_in"] + first[-1]).to(torch.int32)]


def _plain_norm_rope(x, weight, s):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rot = s["case"]["rot"]
    cos, sin = s["cos_sin"][s["positions"].long()][:, None].split(rot // 2, -1)
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1).to(torch.bfloat16)


def _plain_rope(s):
    q, k = _plain_norm_rope(s["q"], s["q_weight"], s), _plain_norm_rope(s["k"], s["k_weight"], s)
    if not s["case"]["cache"]:
        return [q, k]
    page, offset = s["slots"] // PAGE, s["slots"] % PAGE
    s["k_cache"][page, offset] = k
    s["v_cache"][page, offset] = s["v"]
    return [q, s["k_cache"], s["v_cache"]]


def _quantise(x, tensor_scale):
    """Codes (0..15) and e4m3 scales of x [..., Dh]: 16 elements share a scale,
    their largest magnitude over 6; ties of the codes go to the even one."""
    x = x.float() / tensor_scale
    blocks = x.unflatten(-1, (-1, 16))
    scales = (blocks.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    r = blocks.abs() / scales.float().unsqueeze(-1)
    code = sum(c.to(torch.uint8) for c in (r > 0.25, r >= 0.75, r > 1.25, r >= 1.75, r > 2.5, r >= 3.5, r > 5))
    code = torch.where(scales.float().unsqueeze(-1) > 0, code, 0) + 8 * torch.signbit(blocks).to(torch.uint8)
    return code.flatten(-2), scales.view(torch.uint8)


def _records(codes, scales, which):
    """The pool's records [blocks, heads, bytes] from codes and scales [blocks, 16, heads, ...]."""
    data = codes[..., 0::2] + 16 * codes[..., 1::2]
    order = (0, 2, 1, 3) if which == "k" else (0, 2, 3, 1)
    return torch.cat([data.permute(*order).flatten(2), scales.permute(*order).flatten(2)], -1).contiguous()


def _values(pool, which, dh, tensor_scale):
    """What records [..., heads, bytes] stand for: [..., 16, heads, Dh] in 32 bits."""
    data, scales = pool.split([PAGE * dh // 2, PAGE * dh // 16], -1)
    if which == "k":
        data, scales = data.unflatten(-1, (PAGE, dh // 2)), scales.unflatten(-1, (PAGE, dh // 16))
    else:
        data, scales = data.unflatten(-1, (dh // 2, PAGE)).mT, scales.unflatten(-1, (dh // 16, PAGE)).mT
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=pool.device)
    levels = torch.cat([levels, -levels])
    value = levels[torch.stack([data & 15, data >> 4], -1).flatten(-2).long()]
    factor = scales.contiguous().view(torch.float8_e4m3fn).float() * tensor_scale
    value = (value.unflatten(-1, (-1, 16)) * factor.unsqueeze(-1)).flatten(-2)
    return value.transpose(-3, -2)


def _plain_quant(s):
    dh = s["case"]["dh"]
    page, offset = s["slots"] // PAGE, s["slots"] % PAGE
    for name, x in (("k", s["key"]), ("v", s["value"])):
        codes, scales = _quantise(x, s[name + "_scale"])
        data = codes[..., 0::2] + 16 * codes[..., 1::2]
        pool_data, pool_scales = s[name + "_pool"].split([PAGE * dh // 2, PAGE * dh // 16], -1)
        if name == "k":
            pool_data.unflatten(-1, (PAGE, -1))[page, :, offset] = data
            pool_scales.unflatten(-1, (PAGE, -1))[page, :, offset] = scales
        else:
            pool_data.unflatten(-1, (-1, PAGE))[page, :, :, offset] = data
            pool_scales.unflatten(-1, (-1, PAGE))[page, :, :, offset] = scales
    counts = (s["seq_lens"].long() + PAGE - 1) // PAGE
    offsets = _exclusive(counts)
    col = torch.arange(s["block_tables"].shape[1], device=counts.device)
    used = col < counts[:, None]
    ids = s["block_tables"].long()[used]
    return [_values(s["k_pool"][ids], "k", dh, s["k_scale"]).to(torch.bfloat16),
            _values(s["v_pool"][ids], "v", dh, s["v_scale"]).to(torch.bfloat16),
            torch.where(used, offsets[:-1, None] + col, -1).to(torch.int32), offsets.to(torch.int32)]


def _plain_attention(s):
    """Causal softmax attention over the padded contexts."""
    case, lens = s["case"], s["seq_lens"].long()
    hq, hkv, dh, new = case["hq"], case["hkv"], case["dh"], case["new"]
    batch = lens.numel()
    columns = _pages(s["max_seq_len"])
    col = torch.arange(columns, device=lens.device)
    ids = torch.where(col < ((lens + PAGE - 1) // PAGE)[:, None], s["block_tables"][:, :columns].long(), 0)
    k = _values(s["k_pool"][ids], "k", dh, s["k_scale"]).flatten(1, 2)
    v = _values(s["v_pool"][ids], "v", dh, s["v_scale"]).flatten(1, 2)
    q = s["q"].float().view(batch, new, hkv, hq // hkv, dh).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    limit = (lens[:, None] - new + torch.arange(new, device=lens.device)).repeat(1, hq // hkv)
    seen = torch.arange(columns * PAGE, device=lens.device) <= limit[..., None]
    scores = scores.masked_fill(~seen[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = v.permute(0, 2, 1, 3).masked_fill((torch.arange(columns * PAGE, device=lens.device) >= lens[:, None])[:, None, :, None], 0)
    out = torch.matmul(p, v) / total
    out = out.unflatten(2, (hq // hkv, new)).permute(0, 3, 1, 2, 4).reshape(batch * new, hq, dh)
    lse = (top + torch.log(total)).squeeze(-1).unflatten(2, (hq // hkv, new)).permute(0, 3, 1, 2).reshape(batch * new, hq)
    return [out.to(torch.bfloat16), lse]


# ----------------------------------------------------------- in 64 bits -----

def exact(case, seed):
    if case["op"] == "metadata":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    return _exact_quant(s) if case["op"] == "quant" else _exact_attention(s)


def _exact_rope(s):
    case = s["case"]
    half = case["rot"] // 2
    done = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double().clone()
        if w is not None:
            y /= torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + s["eps"])
            y *= w.double()
        row = s["cos_sin"].double()[s["positions"].long()].unsqueeze(1)
        z = torch.complex(row[..., :half], row[..., half:])
        first = torch.arange(half, device=y.device) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        turned = torch.complex(y[..., first], y[..., second]) * z
        y[..., first], y[..., second] = turned.real, turned.imag
        done.append(y)
    if not case["cache"]:
        return done
    pools = []
    for pool, x in ((s["k_cache"], done[1]), (s["v_cache"], s["v"].double())):
        flat = pool.double().flatten(0, 1)
        flat[s["slots"]] = x
        pools.append(flat.view(pool.shape))
    return [done[0]] + pools


def _e4m3(byte):
    """The value of an e4m3 byte, from its fields."""
    table = [(8 + b % 8) / 8 * 2.0 ** (b // 8 - 7) if b > 7 else b / 8 * 2.0 ** -6 for b in range(127)] + [math.nan]
    table = torch.tensor(table + [-x for x in table], dtype=torch.float64, device=byte.device)
    return table[byte.long()]


def _exact_pages(s, ids, which):
    """Pages `ids` of the pool as [pages, 16, heads, Dh] in 64 bits."""
    dh = s["case"]["dh"]
    rec = s[which + "_pool"][ids]
    n, hkv = rec.shape[:2]
    low = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=rec.device)
    pair = torch.stack([low.repeat(16), low.repeat_interleave(16)], -1)  # by byte: (low half, high half)
    shape = (n, hkv, PAGE, dh // 2) if which == "k" else (n, hkv, dh // 2, PAGE)
    body = rec[..., :PAGE * dh // 2].reshape(shape)
    factor = _e4m3(rec[..., PAGE * dh // 2:]).reshape(shape[:2] + tuple(x // 8 if x == dh // 2 else x for x in shape[2:]))
    if which == "v":
        body, factor = body.swapaxes(2, 3), factor.swapaxes(2, 3)
    x = pair[body.long()].reshape(n, hkv, PAGE, dh) * factor.repeat_interleave(16, -1)
    return x.permute(0, 2, 1, 3) * s[which + "_scale"]


def _nearest(x, grid):
    """Index of the grid value nearest to x; a tie goes to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(mid, x.contiguous())
    tie = (i < mid.numel()) & (mid[i.clamp(max=mid.numel() - 1)] == x) & (i % 2 == 1)
    return i + tie.long()


def _exact_quant(s):
    dh, dev = s["case"]["dh"], s["key"].device
    steps = _e4m3(torch.arange(127, device=dev))
    levels = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
    ids = [int(p) for row, n in zip(s["block_tables"].tolist(), s["seq_lens"].tolist()) for p in row[:_pages(n)]]
    place = {p: i for i, p in enumerate(ids)}
    at = torch.tensor([place[p] for p in (s["slots"] // PAGE).tolist()], device=dev)
    ids = torch.tensor(ids, device=dev)
    found = []
    for which, x in (("k", s["key"]), ("v", s["value"])):
        pages = _exact_pages(s, ids, which)
        b = (x.double() / s[which + "_scale"]).reshape(x.shape[0], x.shape[1], dh // 16, 16)
        factor = steps[_nearest(b.abs().max(-1).values / 6, steps)].unsqueeze(-1)
        level = levels[_nearest(torch.where(factor > 0, b.abs() / factor, torch.zeros_like(b)), levels)]
        pages[at, s["slots"] % PAGE] = (torch.sign(b) * level * factor).reshape(x.shape) * s[which + "_scale"]
        found.append(pages)
    return found + [None, None]


def _exact_attention(s):
    case = s["case"]
    hq, hkv, new = case["hq"], case["hkv"], case["new"]
    outs, sums = [], []
    for b, n in enumerate(s["seq_lens"].tolist()):
        ids = s["block_tables"][b, :_pages(n)].long()
        k, v = (_exact_pages(s, ids, w).flatten(0, 1)[:n].repeat_interleave(hq // hkv, 1) for w in ("k", "v"))
        q = s["q"][b * new:(b + 1) * new].double()
        t = torch.einsum("ihd,jhd->hij", q, k) * s["scale"]
        t += torch.full((new, n), -math.inf, dtype=torch.float64, device=t.device).triu(n - new + 1)
        sums.append(torch.logsumexp(t, -1).T)
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(t, -1), v))
    return [torch.cat(outs), torch.cat(sums)]
