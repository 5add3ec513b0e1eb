"""Calls of the 4-bit cache that its description allows beside the ordinary
ones: more tiles than one fold sums by itself, the largest batches, pools in
head-major order and past 2^32 bytes, results in pinned host memory, page
bounds above what the lengths allow, tokens before the first request."""
import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_quant_attention import Case, _same
from tests.test_gpu_quant_cache import _table, _tokens

pytestmark = pytest.mark.gpu


def _alone(c, b, **kw):
    """Request b of the case by itself."""
    lo, hi = int(c.starts[b]), int(c.starts[b + 1])
    return c.run(q=c.q[lo:hi], block_tables=c.bt[b:b + 1].contiguous(), seq_lens=c.sl[b:b + 1].contiguous(),
                 query_start_loc=torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"), max_s=c.lens[b], **kw), (lo, hi)


@pytest.mark.parametrize("dh,hq,hkv,new,lens", [(128, 4, 2, 1, [700, 40, 1300]), (128, 8, 2, 12, [600, 1100]),
                                                (256, 4, 1, 1, [300, 17, 700]), (512, 4, 1, 2, [150, 400])])
def test_more_tiles_than_a_fold_sums_by_itself(dh, hq, hkv, new, lens):
    n = 402 // len(lens) * len(lens)
    c = Case(lens * (n // len(lens)), new, hq, hkv, dh, seed=dh + new)
    out, lse = c.run()
    assert "direct" in pa.last_launch_info() and pa.check_errors() == (pa.PA_OK, -1)
    for b in (0, 1, 2, 255, 256, 257, n - 2, n - 1):
        (o, l), (lo, hi) = _alone(c, b)
        assert _same(o, out[lo:hi]) and _same(l, lse[lo:hi]), b
    pages = sum(-(-x // 16) for x in c.lens)
    o, l = c.run(max_pages=pages)
    assert _same(o, out) and _same(l, lse)
    o, l = c.run(max_pages=10 ** 9)
    assert _same(o, out) and _same(l, lse)
    assert pa.check_errors() == (pa.PA_OK, -1)
    o, l = c.run(max_pages=pages - 1)
    assert bool(o.isnan().all()) and bool(l.isnan().all())
    assert pa.check_errors() == (pa.PA_ERR_WORKSPACE, pages)


def test_the_largest_batch():
    lens = [1 + (29 * i) % 700 for i in range(2048)]
    new = [0 if i % 7 == 3 else 1 for i in range(2048)]
    c = Case(lens, new, 2, 1, 128, seed=31)
    out, lse = c.run()
    assert "direct" in pa.last_launch_info() and pa.check_errors() == (pa.PA_OK, -1)
    for b in (0, 1, 500, 1024, 2045, 2047):
        (o, l), (lo, hi) = _alone(c, b, max_q=1)
        assert _same(o, out[lo:hi]) and _same(l, lse[lo:hi]), b


def test_the_largest_read_back():
    lens = [(5 * i) % 40 for i in range(8192)]
    total = sum(-(-n // 16) for n in lens)
    cache = pa.new_quant_cache(total, 1, 128)
    g = torch.Generator().manual_seed(4)
    for p in (cache.k_pool, cache.v_pool):
        p.copy_(torch.randint(0, 0x70, tuple(p.shape), generator=g, dtype=torch.uint8))
    bt, sl = _table(lens, total, 3, 7)
    ko, vo = torch.zeros(2, total, 16, 1, 128, dtype=torch.bfloat16, device="cuda").unbind(0)
    ct, co = torch.empty_like(bt), torch.empty(8193, dtype=torch.int32, device="cuda")
    pa.dequantize_kv(cache, bt, sl, ko, vo, ct, co)
    assert pa.check_errors() == (pa.PA_OK, -1)
    off = np.concatenate([[0], np.cumsum([-(-n // 16) for n in lens])])
    assert np.array_equal(co.cpu().numpy(), off)
    # the same pages, asked for as one request's
    ids = torch.cat([bt[b, :-(-n // 16)] for b, n in enumerate(lens)]).view(1, -1).contiguous()
    k1, v1 = torch.zeros(2, total, 16, 1, 128, dtype=torch.bfloat16, device="cuda").unbind(0)
    pa.dequantize_kv(cache, ids, torch.tensor([total * 16], dtype=torch.int32, device="cuda"), k1, v1,
                     torch.empty_like(ids), torch.empty(2, dtype=torch.int32, device="cuda"))
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _same(ko, k1) and _same(vo, v1)


@pytest.mark.parametrize("new,hq,kind", [(1, 8, "direct"), (60, 64, "read-back")])
def test_head_major_pools(new, hq, kind):
    hkv, dh = 8, 128
    c = Case([700, 90], new, hq, hkv, dh, seed=33)
    out, lse = c.run(max_q=max(c.new))
    assert kind in pa.last_launch_info()
    old = c.cache
    pools = torch.zeros(2, hkv, old.num_blocks, 9 * dh, dtype=torch.uint8, device="cuda").transpose(1, 2)
    pools[0].copy_(old.k_pool)
    pools[1].copy_(old.v_pool)
    c.cache = pa.QuantCache(pools[0], pools[1], dh)
    o, l = c.run()
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _same(o, out) and _same(l, lse)
    # and the write
    k, v = _tokens(40, hkv, dh, 2)
    slots = torch.randperm(old.num_blocks * 16, generator=torch.Generator().manual_seed(3))[:40].cuda()
    for cache in (old, c.cache):
        pa.reshape_and_cache_quant(k, v, cache, slots)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert torch.equal(pools[0], old.k_pool) and torch.equal(pools[1], old.v_pool)


def test_attention_over_a_pool_past_two_to_the_32_bytes():
    hkv, dh = 8, 512
    c = Case([300, 45], 1, 8, hkv, dh, seed=34)
    out, lse = c.run()
    blocks = 2 ** 32 // (hkv * 9 * dh) + c.cache.num_blocks + 1
    kp = torch.zeros(blocks, hkv, 9 * dh, dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    shift = blocks - c.cache.num_blocks
    kp[shift:].copy_(c.cache.k_pool)
    vp[shift:].copy_(c.cache.v_pool)
    c.cache = pa.QuantCache(kp, vp, dh)
    bt = torch.where(c.bt < 2 ** 30, c.bt + shift, c.bt)
    o, l = c.run(block_tables=bt)
    assert "direct" in pa.last_launch_info() and pa.check_errors() == (pa.PA_OK, -1)
    assert _same(o, out) and _same(l, lse)


@pytest.mark.parametrize("lens,new,hq,hkv", [([700, 90], 1, 8, 2), ([400, 90] * 6, 60, 8, 2)])
def test_results_in_pinned_host_memory(lens, new, hq, hkv):
    c = Case(lens, new, hq, hkv, 128, seed=35)
    out, lse = c.run()
    o, l = torch.zeros(out.shape, dtype=out.dtype).pin_memory(), torch.zeros(lse.shape).pin_memory()
    c.run(out=o, lse=l)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _same(o, out.cpu()) and _same(l, lse.cpu())


@pytest.mark.parametrize("new,hq,hkv,kind", [(1, 8, 2, "direct"), (9, 8, 2, "direct"), (60, 64, 16, "read-back")])
def test_tokens_before_the_first_request_and_between_requests(new, hq, hkv, kind):
    """Requests read ranges of their own; what is in none of them is left alone."""
    c = Case([300, 200, 150], new, hq, hkv, 128, seed=36)
    out, lse = c.run()
    assert kind in pa.last_launch_info()
    q = torch.cat([c.q[:3], c.q])
    o, l = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    c.run(q=q, query_start_loc=c.qs + 3, out=o, lse=l)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _same(o[3:], out) and _same(l[3:], lse)
    assert bool((o[:3] == 7).all()) and bool((l[:3] == 7).all())
