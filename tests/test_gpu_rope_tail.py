"""Elements from rot_dim on are not rotated: without a norm they come out bit
for bit, whatever their neighbours hold."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.helpers import bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dh,rot", [(128, 16), (128, 64), (128, 80), (128, 112), (256, 32), (256, 192), (512, 48),
                                    (512, 272), (512, 496)])
def test_unrotated_elements_pass_unchanged(dh, rot, interleaved):
    T, hq, hkv = 21, 5, 2
    g = torch.Generator().manual_seed(dh + rot)
    q, k = (torch.randn(T, h, dh, generator=g).to(torch.bfloat16) for h in (hq, hkv))
    for x in (q, k):
        tail = x[..., rot:]
        kind = torch.randint(0, 8, tail.shape, generator=g)
        for i, value in enumerate((0.0, -0.0, float("inf"), -float("inf"), float("nan"))):
            tail[kind == i] = value
    q, k = q.cuda(), k.cuda()
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32).cuda()
    table = pa.rope_table(300, rot, device="cuda")
    qo, ko = pa.qk_norm_rope(q, k, pos, table, interleaved=interleaved)
    pool = torch.zeros(2, 2, 16, hkv, dh, dtype=torch.bfloat16, device="cuda")
    qc = pa.qk_norm_rope_and_cache(q, k, k, pos, table, pool[0], pool[1], torch.arange(T, device="cuda"),
                                   interleaved=interleaved)
    assert pa.check_errors() == (pa.PA_OK, -1)
    kc = pool[0].flatten(0, 1)[:T]
    for got, x in ((qo, q), (ko, k), (qc, q), (kc, k)):
        a, b = got[..., rot:], x[..., rot:]
        nan = b.isnan()
        assert torch.equal(a.isnan(), nan)
        assert (bits(a[~nan]) == bits(b[~nan])).all()
        assert bool(got[..., :rot].isfinite().all())
