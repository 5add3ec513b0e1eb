"""pa_release_pages refused for want of room: every count is what it was, also of
pages that were given up more often than they had owners."""
import numpy as np
import pytest

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_pages import State, _release

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("times", [2, 3, 7])
def test_a_page_given_up_too_often_and_no_room(times, in_place):
    """One row names a page of one owner `times` times; the stack below the cursor
    holds fewer pages than the call frees."""
    s = State([100, 90])
    s.tables[1, :times - 1] = s.tables[1, 5]
    s.cursor = 4
    _, bad = _release(s, [0, 0], in_place)
    assert bad == ("request", 1)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("room", [0, 1, 8, 9, 12])
def test_shared_pages_given_up_too_often(room, in_place):
    """Two pages of three owners that two of them name twice more each.  Nine pages
    lose their last owner (13 less four that no row names any more)."""
    s = State([100, 90, 64], groups=3, common=2)
    s.tables[0, 4:6] = s.tables[0, 1]
    s.tables[2, 2:4] = s.tables[2, 0]
    s.cursor = room
    _, bad = _release(s, [0, 0, 0], in_place, loose=True)
    assert bad[0] == "request"


@pytest.mark.parametrize("in_place", [False, True])
def test_many_references_given_up_too_often_and_no_room(in_place):
    """More references than the lanes' registers hold, a tenth of the columns naming
    a page of the same row again."""
    s = State([360000] * 8, groups=2, common=1500, cols=22501)
    rng = np.random.default_rng(3)
    for b in range(8):
        cols = rng.choice(22500, 2250, replace=False)
        s.tables[b, cols] = s.tables[b, rng.choice(22500, 2250)]
    s.cursor = 1000
    _, bad = _release(s, [0, 0, 16 * 1600, 0, -1, 0, 160000, 0], in_place)
    assert bad[0] == "request"


@pytest.mark.parametrize("in_place", [False, True])
def test_a_release_that_fits_after_one_that_did_not(in_place):
    s = State([100, 90])
    s.tables[1, 4] = s.tables[1, 3]
    cursor, s.cursor = s.cursor, 3
    _release(s, [0, 0], in_place)
    s.cursor = cursor
    _, bad = _release(s, [0, 0], in_place, loose=True)
    assert bad == ("request", 1)
    assert pa.check_errors() == (pa.PA_OK, -1)
