"""pa_paged_attention_quant on the GPU.

Few rows (the direct kernel) against softmax attention in 64 bits over the
values that the pool stands for.  Tolerances, per element:
  scores: d = Dh products of exact factors summed in fp32 (at most Dh + 2
    roundings of 2^-24 of the sum of magnitudes, doubled for the chain's
    order), q's scaling (2^-25 of its largest element, covered by one more
    rounding), the change to log2 units and back (4 roundings):
    (2*Dh + 8) * 2^-24 * reach, plus 2^-21 for the exponential;
  out: 2^-8 |out| (rounding to BF16) + (2^-11 (p rounded to f16) + 2 d + 2^-18
    (sums, folds and their factors)) * spread + 2^-40 * n * max |v|: p is held
    as f16 times 2^15, whose smallest steps are 2^-24, so each of the n keys'
    p is off by at most half a step, 2^-25 * 2^-15 of the row's largest (1, and
    the sum of p is at least that);
  lse: d + 2^-18 + 2^-22 |lse|.
More rows in larger calls: bit for bit pa_paged_attention over the read-back
pool."""
import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import step_reference as ref
from tests.helpers import bits, bits_to_f64

pytestmark = pytest.mark.gpu


def _f64(t):
    return bits_to_f64(bits(t))


def _cache(blocks, hkv, dh, seed, k_scale=1.0, v_scale=1.0, interleaved=True):
    """A pool of normal values, quantised by the reference."""
    g = torch.Generator().manual_seed(seed)
    pools = []
    for which, s in (("k", k_scale), ("v", v_scale)):
        x = torch.randn(blocks, 16, hkv, dh, generator=g).to(torch.bfloat16).double().numpy() * s
        codes, sc = ref.quantise(x, s)
        data = codes[..., 0::2] | codes[..., 1::2] << 4
        order = (0, 2, 1, 3) if which == "k" else (0, 2, 3, 1)
        pools.append(np.concatenate([a.transpose(order).reshape(blocks, hkv, -1) for a in (data, sc)], -1))
    both = torch.from_numpy(np.stack(pools, 1 if interleaved else 0)).cuda()
    return pa.QuantCache(*(both.unbind(1) if interleaved else both.unbind(0)), dh, k_scale, v_scale)


class Case:
    def __init__(self, lens, new, hq, hkv, dh, seed=0, spare=3, std=1.0, **kw):
        new = [new] * len(lens) if isinstance(new, int) else new
        total = sum(-(-n // 16) for n in lens)
        self.lens, self.new, self.hq, self.hkv, self.dh = lens, new, hq, hkv, dh
        self.cache = _cache(total + spare, hkv, dh, seed, **kw)
        rng = np.random.default_rng(seed)
        perm, at = rng.permutation(total + spare), 0
        self.tables = np.full((len(lens), max(1, max(-(-n // 16) for n in lens))), 2**31 - 1, np.int32)
        for b, n in enumerate(lens):
            m = -(-n // 16)
            self.tables[b, :m] = perm[at:at + m]
            at += m
        g = torch.Generator().manual_seed(seed + 1)
        self.q = (std * torch.randn(sum(new), hq, dh, generator=g)).to(torch.bfloat16).cuda()
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.scale = 1 / dh ** 0.5
        self.bt, self.sl, self.qs = (torch.from_numpy(np.asarray(x, np.int32)).cuda()
                                     for x in (self.tables, lens, self.starts))

    def run(self, max_q=None, max_s=None, **kw):
        a = dict(q=self.q, block_tables=self.bt, seq_lens=self.sl, query_start_loc=self.qs)
        extra = {k: kw.pop(k) for k in list(kw) if k in ("out", "lse", "workspace", "max_pages", "stream")}
        a.update(kw)
        return pa.paged_attention_quant(a["q"], self.cache, a["block_tables"], a["seq_lens"], a["query_start_loc"],
                                        self.scale, max_q or max(self.new), max_s or max(self.lens), **extra)

    def reference(self):
        k = ref.pool_values(self.cache.k_pool.cpu().numpy(), "k", self.dh, self.cache.struct.k_scale)
        v = ref.pool_values(self.cache.v_pool.cpu().numpy(), "v", self.dh, self.cache.struct.v_scale)
        return ref.attention(_f64(self.q), k, v, self.tables, self.lens, self.starts, self.scale)

    def check(self, out, lse):
        w_out, w_lse, spread, reach = self.reference()
        d = (2 * self.dh + 8) * 2.0 ** -24 * reach + 2.0 ** -21
        v = ref.pool_values(self.cache.v_pool.cpu().numpy(), "v", self.dh, self.cache.struct.v_scale)
        tol = 2.0 ** -8 * np.abs(w_out) + (2.0 ** -11 + 2 * d[..., None] + 2.0 ** -18) * spread \
            + 2.0 ** -40 * max(self.lens) * np.abs(v).max()
        err = np.abs(_f64(out) - w_out)
        assert (err <= tol).all(), float((err / tol).max())
        if lse is not None:
            e, t = np.abs(lse.cpu().double().numpy() - w_lse), d + 2.0 ** -18 + 2.0 ** -22 * np.abs(w_lse)
            assert (e <= t).all(), float((e / t).max())


def _same(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                       b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


@pytest.mark.parametrize("lens,new,hq,hkv,dh", [
    ([1], 1, 1, 1, 128), ([16], 1, 8, 2, 128), ([17, 1, 128, 129, 255, 256, 257], 1, 8, 2, 128),
    ([700, 513], 1, 7, 1, 128), ([300, 40], 1, 16, 2, 128), ([300, 5, 129], 5, 8, 2, 128), ([64, 600], 4, 8, 1, 128),
    ([530, 31], 2, 32, 2, 128), ([1000], 1, 32, 1, 128), ([2, 3, 300], [2, 1, 3], 8, 2, 128),
    ([90, 257, 1], 1, 8, 2, 256), ([300, 44], 5, 8, 2, 256), ([260], 8, 4, 1, 256), ([131], 3, 10, 2, 256),
    ([200, 33], 1, 16, 2, 512), ([140], 2, 16, 2, 512), ([150], 4, 4, 1, 512), ([4097], 1, 4, 1, 512),
    ([5, 9, 40], [0, 1, 2], 4, 4, 128),
    # two tiles of tokens
    ([300, 77, 9, 1040], [8, 5, 1, 3], 8, 1, 128), ([700, 40], 8, 28, 4, 128), ([530, 31], [16, 9], 8, 2, 128),
    ([64, 600], 2, 32, 1, 128), ([300, 44], [9, 16], 8, 2, 256), ([140, 33], [6, 8], 8, 2, 512), ([9], 9, 4, 1, 128),
    # more tiles, in small calls
    ([300, 77], 77, 8, 2, 128), ([513, 40, 1030], [17, 40, 33], 8, 2, 128), ([200], 20, 16, 2, 256),
    ([150, 64], 50, 16, 2, 512), ([100, 1, 30, 600], [70, 1, 0, 5], 4, 4, 128), ([700], 10, 7, 1, 256)])
def test_direct_matches_formula(lens, new, hq, hkv, dh):
    c = Case(lens, new, hq, hkv, dh, seed=len(lens) + dh + hq, k_scale=0.5, v_scale=2.0)
    out, lse = c.run()
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert "direct" in pa.last_launch_info()
    c.check(out, lse)


def test_direct_long_context_and_large_scores():
    c = Case([20011], 1, 8, 2, 128, seed=3, interleaved=False)
    out, lse = c.run()
    c.check(out, lse)
    c = Case([900, 333], 2, 4, 1, 128, seed=4, std=300.0)   # one key takes nearly everything
    out, lse = c.run()
    c.check(out, lse)
    c = Case([900, 333], 2, 4, 1, 128, seed=5, std=1e-6)    # uniform weights
    out, lse = c.run()
    c.check(out, lse)
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_rows_do_not_depend_on_batch_bounds_or_splits():
    """Every request alone, with other bounds, at another place of a larger
    batch: the same bits."""
    lens = [7168, 700, 4171, 513, 31, 1, 256, 1300]
    c = Case(lens, 1, 8, 2, 128, seed=6)
    out, lse = c.run()
    wide_out, wide_lse = c.run(max_q=6, max_s=20000)        # 24 rows' worth of bounds
    assert _same(out, wide_out) and _same(lse, wide_lse)
    for b, n in enumerate(lens):
        o, l = c.run(q=c.q[b:b + 1], block_tables=c.bt[b:b + 1].contiguous(), seq_lens=c.sl[b:b + 1].contiguous(),
                     query_start_loc=torch.tensor([0, 1], dtype=torch.int32, device="cuda"), max_s=n)
        assert _same(o, out[b:b + 1]) and _same(l, lse[b:b + 1]), n
    many = [i % 8 for i in range(75)]
    idx = torch.tensor(many, device="cuda")
    o, l = c.run(q=c.q[idx], block_tables=c.bt[idx], seq_lens=c.sl[idx],
                 query_start_loc=torch.arange(76, dtype=torch.int32, device="cuda"))
    assert _same(o, out[idx]) and _same(l, lse[idx])
    assert pa.check_errors() == (pa.PA_OK, -1)


@pytest.mark.parametrize("new,hq,hkv,dh", [(5, 8, 2, 128), (8, 2, 2, 128), (2, 16, 1, 128), (5, 8, 2, 256), (4, 8, 2, 512),
                                              (12, 8, 2, 128), (8, 7, 1, 128), (11, 8, 2, 256), (6, 8, 2, 512),
                                              (33, 8, 2, 128), (20, 16, 2, 256), (9, 8, 1, 512)])
def test_drafted_tokens_equal_single_steps_in_bits(new, hq, hkv, dh):
    """Token i of a request's `new` tokens equals the single-token call at its length."""
    c = Case([1030, 258], new, hq, hkv, dh, seed=7)
    out, lse = c.run()
    for i in range(new):
        rows = torch.tensor([i, new + i], device="cuda")
        o, l = c.run(q=c.q[rows], seq_lens=c.sl - (new - 1 - i), max_q=1,
                     query_start_loc=torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"))
        assert _same(o, out[rows]) and _same(l, lse[rows]), i


@pytest.mark.parametrize("dh,hq,hkv,new", [(128, 8, 2, 1), (256, 8, 2, 3), (512, 8, 2, 2)])
def test_rows_of_a_large_batch_equal_those_of_small_calls(dh, hq, hkv, new):
    """The folding kernel splits rows between warps only in small calls, and
    the deal of the chunks depends on the batch: no bit may."""
    lens = [700, 33, 5000, 300] * 12
    c = Case(lens, new, hq, hkv, dh, seed=dh + 1)
    out, lse = c.run()
    for b in (0, 2, 7, 46):
        rows = torch.arange(b * new, (b + 1) * new, device="cuda")
        o, l = c.run(q=c.q[rows], block_tables=c.bt[b:b + 1].contiguous(), seq_lens=c.sl[b:b + 1].contiguous(),
                     query_start_loc=torch.tensor([0, new], dtype=torch.int32, device="cuda"), max_s=lens[b])
        assert _same(o, out[rows]) and _same(l, lse[rows]), b
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_bytes_past_the_length_and_unseen_nans_do_not_matter():
    c = Case([37, 130, 20], [3, 2, 1], 8, 2, 128, seed=8)
    out, lse = c.run()
    for b, n in enumerate(c.lens):
        page = int(c.tables[b, (n - 1) // 16])
        codes, sc = c.cache.k_pool[page], c.cache.v_pool[page]
        for tok in range(n % 16 or 16, 16):
            codes[:, 8 * 128:].view(2, 16, 8)[:, tok] = 0x7F
            sc[:, 8 * 128:].view(2, 8, 16)[:, :, tok] = 0x7F
    o, l = c.run()
    assert _same(o, out) and _same(l, lse)
    # the newest token of request 0 holds NaN in one V block and one K block:
    # its two older rows do not see it
    page = int(c.tables[0, 2])
    c.cache.v_pool[page][:, 8 * 128:].view(2, 8, 16)[1, 3, 4] = 0x7F
    o, l = c.run()
    assert _same(o[:2], out[:2]) and _same(o[3:], out[3:]) and _same(l, lse)
    bad = o[2].isnan()
    assert bool(bad[4:, 48:64].all()) and int(bad.sum()) == 4 * 16
    c.cache.k_pool[page][:, 8 * 128:].view(2, 16, 8)[0, 4, 2] = 0x7F
    o, l = c.run()
    assert _same(o[:2], out[:2]) and _same(l[:2], lse[:2])
    assert bool(o[2, :4].isnan().all()) and bool(l[2, :4].isnan().all()) and not bool(l[2, 4:].isnan().any())
    assert pa.check_errors() == (pa.PA_OK, -1)


@pytest.mark.parametrize("new,hq,hkv,kind", [(1, 8, 2, "direct"), (10, 8, 2, "direct"), (40, 8, 2, "direct"),
                                             (40, 64, 16, "read-back")])
def test_bad_metadata_gives_nan_rows_and_leaves_the_rest(new, hq, hkv, kind):
    c = Case([300, 200, 150], new, hq, hkv, 128, seed=9)
    out, lse = c.run()
    assert kind in pa.last_launch_info()
    bt = c.bt.clone()
    bt[1, 3] = 10**6
    fill = torch.full_like(out, 7.0)
    o, l = c.run(block_tables=bt, out=fill.clone())
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 1)
    assert bool(o[new:2 * new].isnan().all()) and _same(o[:new], out[:new]) and _same(o[2 * new:], out[2 * new:])
    o, l = c.run(seq_lens=torch.tensor([300, 0, 150], dtype=torch.int32, device="cuda"), out=fill.clone())
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 1)
    assert bool(o[new:2 * new].isnan().all()) and bool(l[new:2 * new].isnan().all())
    assert _same(o[:new], out[:new]) and _same(o[2 * new:], out[2 * new:])
    # a request past the bound of lengths
    o, l = c.run(max_s=250, out=fill.clone())
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 0)
    assert bool(o[:new].isnan().all()) and _same(o[new:], out[new:])
    # rows that no request owns stay as they are
    tail = torch.full((3 * new + 2, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.cat([c.q, c.q[:2]])
    o, _ = c.run(q=q, out=tail)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _same(o[:3 * new], out) and bool((o[3 * new:] == 7).all())


@pytest.mark.parametrize("lens,new,hq,hkv,dh", [([300, 77] * 4, 77, 8, 2, 128),
                                                ([513, 40, 1030] * 6, [17, 40, 33] * 6, 8, 2, 128),
                                                ([200] * 16, 20, 16, 2, 256), ([150, 64] * 2, 50, 16, 2, 512),
                                                ([40, 3], 1, 128, 1, 128)])
def test_more_rows_equal_bf16_attention_on_the_read_back_pool(lens, new, hq, hkv, dh):
    c = Case(lens, new, hq, hkv, dh, seed=dh, k_scale=2.0, v_scale=0.25)
    out, lse = c.run()
    assert "read-back" in pa.last_launch_info()
    total = sum(-(-n // 16) for n in lens)
    ko, vo = torch.empty(2, total, 16, hkv, dh, dtype=torch.bfloat16, device="cuda").unbind(0)
    ct, co = torch.empty_like(c.bt), torch.empty(len(lens) + 1, dtype=torch.int32, device="cuda")
    pa.dequantize_kv(c.cache, c.bt, c.sl, ko, vo, ct, co)
    o, l = pa.paged_attention(c.q, ko, vo, ct, c.sl, c.qs, c.scale, max(c.new), max(lens))
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _same(out, o) and _same(lse, l)
    o, l = c.run(max_pages=total)
    assert pa.check_errors() == (pa.PA_OK, -1) and _same(out, o)
    if total > 1:
        o, l = c.run(max_pages=total - 1)
        assert pa.check_errors() == (pa.PA_ERR_WORKSPACE, total)
        assert bool(o.isnan().all()) and bool(l.isnan().all())


def test_errors_and_nans_seen_by_the_second_tile_only():
    """Ten tokens of four query heads to a KV head: tiles of five tokens."""
    c = Case([1037, 200], 10, 8, 2, 128, seed=16)
    out, lse = c.run()
    assert "tiles=2" in pa.last_launch_info()
    # the last page's id: every row of the request
    bt = c.bt.clone()
    bt[0, 1036 // 16] = -1
    o, l = c.run(block_tables=bt)
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 0)
    assert bool(o[:10].isnan().all()) and bool(l[:10].isnan().all()) and _same(o[10:], out[10:])
    # more tokens than the bound allows: every row, and no other
    o, l = c.run(query_start_loc=torch.tensor([0, 13, 20], dtype=torch.int32, device="cuda"), max_q=10)
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 0)
    assert bool(o[:13].isnan().all()) and bool(l[:13].isnan().all()) and not bool(o[13:].isnan().any())
    # a NaN scale of V at a key that only the last two tokens see
    page, tok = int(c.tables[0, 1035 // 16]), 1035 % 16
    c.cache.v_pool[page, 0, 8 * 128 + 3 * 16 + tok] = 0x7F
    o, l = c.run()
    want = torch.zeros_like(o, dtype=torch.bool)
    want[8:10, :4, 48:64] = True
    assert torch.equal(o.isnan(), want) and _same(l, lse)
    assert _same(o[~want], out[~want])
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_unseen_nans_where_groups_follow_one_another_in_a_cta():
    """Far more groups than CTAs, of lengths in turn short and long: a NaN that
    only a request's last token sees reaches that row alone."""
    n = 300
    c = Case([40, 500] * (n // 2), 2, 8, 2, 128, seed=18)
    out, lse = c.run()
    for b, length in enumerate(c.lens):
        page, tok = int(c.tables[b, (length - 1) // 16]), (length - 1) % 16
        c.cache.v_pool[page, 1, 8 * 128 + 5 * 16 + tok] = 0x7F
    want = torch.zeros_like(out, dtype=torch.bool)
    want[1::2, 4:, 80:96] = True
    for _ in range(5):
        o, l = c.run()
        assert torch.equal(o.isnan(), want) and _same(l, lse)
        assert _same(o[~want], out[~want])
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_one_workspace_serves_calls_of_different_bounds():
    a = Case([7168, 513], 1, 8, 2, 128, seed=11)
    b = Case([400, 90] * 6, 60, 8, 2, 128, seed=12)
    ra, rb = a.run(), b.run()
    assert "read-back" in pa.last_launch_info()
    n = max(pa.quant_workspace_size(2, 8, 2, 128, 1, 7168), pa.quant_workspace_size(12, 8, 2, 128, 60, 400))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for c, r in ((a, ra), (b, rb)):
            o, l = c.run(workspace=ws)
            assert _same(o, r[0]) and _same(l, r[1])
    assert pa.check_errors() == (pa.PA_OK, -1)


@pytest.mark.parametrize("new,hq,hkv,kind", [(1, 8, 2, "direct"), (10, 8, 2, "direct"), (20, 8, 2, "direct"),
                                             (20, 64, 16, "read-back")])
def test_a_page_bound_sizes_the_workspace_and_is_enforced(new, hq, hkv, kind):
    c = Case([1500, 20, 700, 513], new, hq, hkv, 128, seed=15)
    out, lse = c.run()
    assert kind in pa.last_launch_info()
    pages = sum(-(-n // 16) for n in c.lens)
    n = pa.quant_workspace_size(4, hq, hkv, 128, new, 1500, pages)
    assert n < pa.quant_workspace_size(4, hq, hkv, 128, new, 1500)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    o, l = c.run(workspace=ws, max_pages=pages)
    assert _same(o, out) and _same(l, lse)
    assert pa.check_errors() == (pa.PA_OK, -1)
    o, l = c.run(workspace=ws, max_pages=pages - 1)
    assert bool(o.isnan().all()) and bool(l.isnan().all())
    assert pa.check_errors() == (pa.PA_ERR_WORKSPACE, pages)
    o, l = c.run(workspace=ws, max_pages=pages)
    assert _same(o, out) and _same(l, lse)


@pytest.mark.parametrize("new,hq,hkv,kind", [(1, 8, 2, "direct"), (40, 64, 16, "read-back")])
def test_calls_on_another_stream_keep_their_own_memory(new, hq, hkv, kind):
    """Results, statistics and scratch that the call allocates belong to its
    stream: what the current stream does meanwhile cannot meet them."""
    c = Case([3000, 513, 90], new, hq, hkv, 128, seed=17)
    out, lse = c.run()
    assert kind in pa.last_launch_info()
    n = pa.quant_workspace_size(3, hq, hkv, 128, new, 3000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        o, l = c.run(stream=side)
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), torch.full_like(o, 3.0)]
        side.synchronize()
        assert _same(o, out) and _same(l, lse)
        del o, l, junk
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_two_graphs_share_a_workspace_and_replay():
    a = Case([3000, 513, 90], 1, 8, 2, 128, seed=13)
    b = Case([400, 90] * 6, 60, 8, 2, 128, seed=14)
    want = [x for c in (a, b) for x in c.run()]
    n = max(pa.quant_workspace_size(3, 8, 2, 128, 1, 3000), pa.quant_workspace_size(12, 8, 2, 128, 60, 400))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    pa.init()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, got = [], []
    for c in (a, b):
        out, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device="cuda")
        torch.cuda.synchronize()
        call = pa.prepare_paged_attention_quant(c.q, c.cache, c.bt, c.sl, c.qs, c.scale, max(c.new), max(c.lens), out,
                                                lse, ws, stream=s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        graphs.append(g)
        got += [out, lse]
    for _ in range(3):
        for t in got:
            t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(_same(x, y) for x, y in zip(got, want))
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_q_slice_no_lse_and_repeat():
    c = Case([500, 90], 1, 8, 2, 128, seed=15)
    out, lse = c.run()
    wide = torch.zeros(2, 12 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    q = wide[:, 8:8 + 1024].view(2, 8, 128)
    q.copy_(c.q)
    o, l = pa.paged_attention_quant(q, c.cache, c.bt, c.sl, c.qs, c.scale, 1, 500, want_lse=False)
    assert l is None and _same(o, out)
    for _ in range(20):
        o, l = c.run()
        assert _same(o, out) and _same(l, lse)


def test_many_requests():
    """More requests than one pass of the request scan, some idle."""
    lens = [1 + (37 * i) % 300 for i in range(600)]
    new = [i % 2 for i in range(600)]
    c = Case(lens, new, 4, 1, 128, seed=16)
    out, lse = c.run()
    assert pa.check_errors() == (pa.PA_OK, -1)
    c.check(out, lse)
