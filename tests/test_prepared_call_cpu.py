"""PreparedCall converts its arguments as a call through the prototypes does."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import build as pa_build
from paged_kv_cache_178_gb300 import pagedattn as pa


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


@pytest.mark.parametrize("head", [1, True, np.int64(1), np.int32(1), torch.tensor(1)])
def test_every_integer_type_that_a_prototype_takes(lib, head):
    """A head number that came out of numpy or torch: the call reaches the
    library, which refuses the null pool."""
    cache = pa.PaKvCache()
    args = (ctypes.byref(cache), head, 0, 1, 0, 1, 0, 0, 1, 0, 0, None)
    assert lib.pa_gather_kv_head(*args) == pa.PA_ERR_INVALID_ARG
    call = pa.PreparedCall(lib.pa_gather_kv_head, args, "pa_gather_kv_head", (cache,))
    for _ in range(2):
        with pytest.raises(pa.PagedAttnError) as e:
            call()
        assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_a_wrong_type_is_refused_when_the_call_is_prepared(lib):
    cache = pa.PaKvCache()
    args = (ctypes.byref(cache), "head", 0, 1, 0, 1, 0, 0, 1, 0, 0, None)
    with pytest.raises((ctypes.ArgumentError, TypeError)):
        pa.PreparedCall(lib.pa_gather_kv_head, args, "pa_gather_kv_head", (cache,))
