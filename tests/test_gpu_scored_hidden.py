"""What a token does not see changes no bit of its result, however large it is."""
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests.test_gpu_scored_attention import _batch

pytestmark = pytest.mark.gpu


def _run(a, rules):
    out, lse = pa.paged_attention_scored(**a, **rules)
    return out, lse, pa.check_errors()


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 1, 256), (4, 1, 512)])
@pytest.mark.parametrize("new", [1, 20, 300])
def test_hidden_keys_of_any_size_change_no_bit(new, heads):
    """Keys behind the length and behind a window, large or zero, and query rows of no
    request: the scores' arithmetic does not depend on them."""
    lens = [700, 333]
    a = _batch(lens, [new] * 2, *heads, seed=4, spread=3.0)
    pad = torch.randn(40, *a["q"].shape[1:], device="cuda").to(torch.bfloat16)
    results = []
    for size in (0.0, 1.0, 1e4, 1e30):
        for b, n in enumerate(lens):
            for j in (x for x in (0, n - new - 101, n - new - 100) if 0 <= x <= n - new - 100):
                a["k_cache"][int(a["block_tables"][b, j // 16]), j % 16] = size
            if n % 16:
                a["k_cache"][int(a["block_tables"][b, n // 16]), n % 16:] = size
        c = dict(a, q=torch.cat([a["q"], pad * size]))
        results.append(_run(c, dict(soft_cap=30.0, window=100)))
    for r in results[1:]:
        n = 2 * new
        assert r[2] == (0, -1)
        assert torch.equal(r[0][:n], results[0][0][:n]) and torch.equal(r[1][:n], results[0][1][:n])
