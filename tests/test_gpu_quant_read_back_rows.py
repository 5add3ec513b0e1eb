"""4-bit attention by way of the read-back: what the pages hold where no row may
look, and a bad block id that only some rows would reach."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_quant_attention import Case, _same

pytestmark = pytest.mark.gpu

SHAPES = [([2000, 300, 77], [1000, 100, 77], 32, 8, 128), ([1500, 40], [1100, 40], 64, 8, 256),
          ([900, 333], [700, 300], 32, 4, 512)]


def _run(c, **kw):
    o, l = c.run(**kw)
    assert "read-back" in pa.last_launch_info(), pa.last_launch_info()
    return o, l


@pytest.mark.parametrize("lens,new,hq,hkv,dh", SHAPES)
@pytest.mark.parametrize("page", ["first", "middle", "last"])
def test_a_bad_block_id_makes_all_rows_of_its_request_nan(lens, new, hq, hkv, dh, page):
    c = Case(lens, new, hq, hkv, dh, seed=21)
    out, lse = _run(c)
    assert pa.check_errors() == (pa.PA_OK, -1)
    n = -(-lens[0] // 16)
    for bad in (c.cache.num_blocks, -1):
        bt = c.bt.clone()
        bt[0, {"first": 0, "middle": n // 2, "last": n - 1}[page]] = bad
        o, l = _run(c, block_tables=bt, out=torch.full_like(out, 7.0), lse=torch.full_like(lse, 7.0))
        assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 0)
        assert bool(o[:new[0]].isnan().all()) and bool(l[:new[0]].isnan().all())
        assert _same(o[new[0]:], out[new[0]:]) and _same(l[new[0]:], lse[new[0]:])


@pytest.mark.parametrize("lens,new,hq,hkv,dh", SHAPES)
def test_bytes_past_the_length_do_not_matter(lens, new, hq, hkv, dh):
    c = Case(lens, new, hq, hkv, dh, seed=22)
    out, lse = _run(c)
    for b, n in enumerate(lens):
        page = int(c.tables[b, (n - 1) // 16])
        codes, sc = c.cache.k_pool[page], c.cache.v_pool[page]
        for tok in range(n % 16 or 16, 16):
            codes[:, 8 * dh:].view(hkv, 16, dh // 16)[:, tok] = 0x7F
            sc[:, 8 * dh:].view(hkv, dh // 16, 16)[:, :, tok] = 0xFF
    o, l = _run(c)
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert _same(o, out) and _same(l, lse)
