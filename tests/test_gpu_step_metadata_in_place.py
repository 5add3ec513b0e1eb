"""Lengths and cursor advancing in place in calls of several CTAs: none may
write over an input before all have read it."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import step_reference as ref
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


def test_a_graph_over_several_ctas_advances_its_own_state():
    """A captured step of 1500 requests, replayed."""
    s = _setup([(13 * i) % 70 for i in range(1500)], [5] * 1500, cursor=0)
    s["new"], s["num_tokens"] = [1] * 1500, 1600
    d = _device(s)
    d["seq_lens"], d["cursor_out"] = d["context_lens"], d["cursor_in"]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pa.init()
    call = pa.prepare_build_step_metadata(**d, stream=st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    assert pa.last_launch_info().endswith("grid=4"), pa.last_launch_info()
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        assert _compare(d, s) is None
        w = ref.step_metadata(s["ctx"], s["new"], s["tables"], s["free"], s["cursor"], s["num_blocks"], 1600)
        s["tables"], s["ctx"], s["cursor"] = w[0], w[3].tolist(), w[5]
    assert pa.check_errors() == (pa.PA_OK, -1)
