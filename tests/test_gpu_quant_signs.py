"""The 4-bit write keeps the sign of every zero, byte for byte against the
64-bit quantiser: zeros of both signs beside other elements, and elements that
round to a zero code."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_quant_cache import _tokens, _write_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0 ** -32, 0.5, 2.0 ** 32])
@pytest.mark.parametrize("T,hkv,dh,consecutive", [(40, 2, 128, True), (23, 8, 128, False), (20, 2, 256, True),
                                                  (17, 1, 512, False)])
def test_zeros_keep_their_signs_beside_other_elements(T, hkv, dh, consecutive, scale):
    k, v = (x.clone() for x in _tokens(T, hkv, dh, T + dh))
    g = torch.Generator().manual_seed(dh)
    for x in (k, v):
        x.mul_(scale)
        kind = torch.randint(0, 6, x.shape, generator=g).cuda()
        x[kind == 0] = 0.0
        x[kind == 1] = -0.0
        # far below the block's scale: a code of zero with the element's sign
        x[kind == 2] *= 2.0 ** -20
        x[kind == 3] *= 2.0 ** -60
        x[0, 0, :16] = -0.0          # a block of one element beside fifteen zeros
        x[0, 0, 7] = scale
        x[1, 0, :16] = 0.0
        x[1, 0, 8] = -scale
    blocks = T // 16 + 3
    slots = torch.arange(5, 5 + T) if consecutive else \
        torch.randperm(blocks * 16, generator=torch.Generator().manual_seed(T))[:T]
    _write_and_check(k, v, slots.cuda(), blocks, "separate", scale, scale)
    assert pa.check_errors() == (pa.PA_OK, -1)


def test_zeros_keep_their_signs_under_a_saturated_scale():
    k, v = (x.clone() for x in _tokens(16, 1, 128, 9))
    for x in (k, v):
        x[:, :, ::16] = 3e38
        x[:, :, 1::16] = -0.0
        x[:, :, 2::16] = 0.0
    _write_and_check(k, v, torch.arange(16, device="cuda"), 1)
    assert pa.check_errors() == (pa.PA_OK, -1)
