"""Lengths and cursor advancing in place in calls of several CTAs: none may
write over an input before all have read it."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_step_metadata import CASES, _compare, _device, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,cursor", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("case,ctas", [("b1025", 4), ("b8192", 8), ("long_prompt", 8), ("b300", 4)])
def test_in_place_over_several_ctas(case, ctas, lens, cursor):
    """Ten runs each: what is read back is what the plain loop gives."""
    s = _setup(*CASES[case], pad=11)
    for _ in range(10):
        d = _device(s)
        if lens:
            d["seq_lens"] = d["context_lens"]
        if cursor:
            d["cursor_out"] = d["cursor_in"]
        pa.build_step_metadata(**d)
        assert pa.last_launch_info().endswith(f"grid={ctas}"), pa.last_launch_info()
        assert pa.check_errors() == (pa.PA_OK, -1)
        assert _compare(d, s) is None


def test_a_large_in_place_step_that_does_not_fit_leaves_the_lengths():
    s = _setup(*CASES["b8192"])
    s["free"] = s["free"][:3]
    d = _device(s)
    d["seq_lens"], d["cursor_out"] = d["context_lens"], d["cursor_in"]
    pa.build_step_metadata(**d)
    assert pa.check_errors()[0] == pa.PA_ERR_WORKSPACE
    assert _compare(d, s) is not None
    assert torch.equal(d["context_lens"].cpu(), torch.tensor(s["ctx"], dtype=torch.int32))
