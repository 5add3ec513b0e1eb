"""Scores far above those of trained models, where a rounding of the score in
32 bits is many units: every result is finite, a row whose best key leads by
more than the scores' error is that key's V to the bit, and a request of one
key always is."""
import numpy as np
import pytest

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import step_reference as ref
from tests.test_gpu_quant_attention import Case, _f64

pytestmark = pytest.mark.gpu


def _winners(c):
    """V of each row's best key [T, Hq, Dh], and whether its lead over the next
    key exceeds what 32-bit scores can blur: twice the bound d of a score's
    error, a rounding of both maxima to log2 units, and 200 (the next key's
    weight is then below exp(-200))."""
    k = ref.pool_values(c.cache.k_pool.cpu().numpy(), "k", c.dh, c.cache.struct.k_scale)
    v = ref.pool_values(c.cache.v_pool.cpu().numpy(), "v", c.dh, c.cache.struct.v_scale)
    q, G = _f64(c.q), c.hq // c.hkv
    best, sure = np.zeros(q.shape), np.zeros(q.shape[:2], bool)
    for b, n in enumerate(c.lens):
        ids = c.tables[b][:-(-n // 16)]
        kk, vv = (x[ids].reshape(-1, c.hkv, c.dh)[:n] for x in (k, v))
        for i in range(c.new[b]):
            t, seen = int(c.starts[b]) + i, n - c.new[b] + i + 1
            for h in range(c.hq):
                z = kk[:seen, h // G] @ q[t, h] * c.scale
                reach = (np.abs(kk[:seen, h // G]) @ np.abs(q[t, h])).max() * c.scale
                d = (2 * c.dh + 8) * 2.0 ** -24 * reach
                order = np.argsort(z)
                best[t, h] = vv[order[-1], h // G]
                lead = np.inf if seen == 1 else z[order[-1]] - z[order[-2]]
                sure[t, h] = lead > 2 * d + 2 * 2.0 ** -23 * reach + 200
    return best, sure


# std of q, k_scale: scores around 1e7, 1e8, 1e9 and 1e11
SIZES = [(1e7, 1.0), (1e8, 1.0), (1e9, 1.0), (1.0, 2.0 ** 32), (16.0, 2.0 ** 32)]


@pytest.mark.parametrize("std,k_scale", SIZES)
@pytest.mark.parametrize("dh,hq,hkv", [(128, 8, 2), (256, 8, 2), (512, 4, 1)])
def test_one_key_gives_its_value(dh, hq, hkv, std, k_scale):
    c = Case([1] * 24, 1, hq, hkv, dh, seed=dh, std=std, k_scale=k_scale)
    out, lse = c.run()
    assert "direct" in pa.last_launch_info()
    assert pa.check_errors() == (pa.PA_OK, -1)
    best, sure = _winners(c)
    assert sure.all() and np.array_equal(_f64(out), best)
    c.check(out, lse)
    assert bool((lse > 0).any()) and bool((lse < 0).any())   # maxima of both signs


@pytest.mark.parametrize("std,k_scale", SIZES)
@pytest.mark.parametrize("lens,new,hq,hkv,dh", [([1300, 333, 17], 1, 8, 2, 128), ([900, 40], 5, 8, 2, 128),
                                                ([600, 250], 2, 8, 2, 256), ([300, 120], 2, 4, 1, 512),
                                                ([700, 90], 8, 7, 1, 128)])
def test_many_keys_give_the_best_one(lens, new, hq, hkv, dh, std, k_scale):
    c = Case(lens, new, hq, hkv, dh, seed=dh + new, std=std, k_scale=k_scale)
    out, lse = c.run()
    assert "direct" in pa.last_launch_info()
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    best, sure = _winners(c)
    assert sure.any() and np.array_equal(_f64(out)[sure], best[sure])
    c.check(out, lse)


@pytest.mark.parametrize("std,k_scale", [(1e7, 1.0), (1e8, 1.0)])
@pytest.mark.parametrize("lens,new,hq,hkv,dh", [([300, 77] * 4, 77, 8, 2, 128), ([200] * 16, 20, 16, 2, 256),
                                                ([150, 64] * 2, 50, 16, 2, 512), ([1, 40, 3], 1, 128, 1, 128)])
def test_the_read_back_gives_the_best_key_too(lens, new, hq, hkv, dh, std, k_scale):
    """P and the result are rounded to BF16 there, half a step (2^-8) each; the
    sums have 2^-14 to spare.  For scores below 2^30: the exponent of the largest
    p is off by half a unit in the last place of the score in log2 units, up to
    64 below 2^31 and 128, where p leaves fp32, from there on."""
    c = Case(lens, new, hq, hkv, dh, seed=dh + new, std=std, k_scale=k_scale)
    out, lse = c.run()
    assert "read-back" in pa.last_launch_info()
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    assert float(lse.abs().max()) < 2.0 ** 30
    best, sure = _winners(c)
    assert sure.any()
    err = np.abs(_f64(out) - best)[sure]
    assert (err <= (2.0 ** -7 + 2.0 ** -14) * np.abs(best[sure])).all(), float(err.max())
