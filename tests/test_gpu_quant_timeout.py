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
