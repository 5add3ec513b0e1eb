"""Waits of the direct 4-bit attention that run out: with the limit at 0 every
wait for copied pages gives up at once, while copies are in flight.  A CTA asks
for no page in place of one that it has not seen land, and ends when the copies
that it asked for have landed; the call latches PA_ERR_TIMEOUT, and the next
one, on the same workspace as it is, gives the reference's bits."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_quant_attention import Case, _same

pytestmark = pytest.mark.gpu

CASES = [([40], 1, 8, 2, 128),                          # one chunk: written without a record
         ([3000, 513, 90], 1, 8, 2, 128),               # a CTA per chunk
         ([700, 33, 5000, 300] * 12, 1, 8, 2, 128),     # several chunks to a CTA
         ([1037, 200], 10, 8, 2, 128),                  # two tiles
         ([700, 2050] * 40, 5, 8, 2, 256), ([300, 1500] * 40, 1, 8, 2, 512)]


def _timed_out(c, **kw):
    prev = pa.set_fold_wait_limit_ns(0)
    try:
        out = c.run(**kw)
        status, _ = pa.check_errors()
    finally:
        assert pa.set_fold_wait_limit_ns(prev) == 0
    assert status == pa.PA_ERR_TIMEOUT
    return out


@pytest.mark.parametrize("lens,new,hq,hkv,dh", CASES)
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(lens, new, hq, hkv, dh):
    c = Case(lens, new, hq, hkv, dh, seed=dh + len(lens))
    out, lse = c.run()
    assert "direct" in pa.last_launch_info() and pa.check_errors() == (pa.PA_OK, -1)
    ws = torch.full((pa.quant_workspace_size(len(lens), hq, hkv, dh, new, max(lens)),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    for _ in range(3):
        _timed_out(c, workspace=ws)
        o, l = c.run(workspace=ws)
        assert pa.check_errors() == (pa.PA_OK, -1)
        assert _same(o, out) and _same(l, lse)


@pytest.mark.parametrize("lens,new,hq,hkv,dh", CASES)
def test_no_row_of_waits_that_ran_out_passes_for_a_result(lens, new, hq, hkv, dh):
    """Requests of several chunks: NaN.  Of one chunk: NaN or not written.  Rows
    that no request owns stay as they are."""
    c = Case(lens, new, hq, hkv, dh, seed=dh + len(lens))
    rows = c.q.shape[0]
    q = torch.cat([c.q, c.q[:1]])
    o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((rows + 1, hq), 7.0, device="cuda")
    # records left by an earlier call, which would pass for results
    ws = torch.zeros(pa.quant_workspace_size(len(lens), hq, hkv, dh, new, max(lens)), dtype=torch.uint8, device="cuda")
    c.run(workspace=ws)
    _timed_out(c, q=q, out=o, lse=l, workspace=ws)
    chunk = {128: 512, 256: 256, 512: 128}[dh]
    for x in (o, l):
        assert bool((x[:rows].isnan() | (x[:rows] == 7)).all()) and bool((x[rows:] == 7).all())
        assert len(lens) == 1 or bool(x[:rows].isnan().any())
        for b, n in enumerate(lens):
            if n > chunk:
                assert bool(x[b * new:(b + 1) * new].isnan().all()), (b, n)
