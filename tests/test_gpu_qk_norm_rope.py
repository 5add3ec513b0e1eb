"""pa_qk_norm_rope and pa_qk_norm_rope_and_cache against the formula in 64 bits.

Tolerance per element: the one rounding to BF16, 2^-8 of the value, plus the
32-bit arithmetic before it: the mean (a tree of at most 16 + 5 additions and
one product, half of whose relative error reaches the root), the root, three
products and the rotation's two products and sum are below 24 roundings of
2^-24 each, relative to |a| + |b| of the pair (size)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import step_reference as ref
from tests.helpers import bits, bits_to_f64

pytestmark = pytest.mark.gpu

FILL = 0x7FC3


def _f64(t):
    return bits_to_f64(bits(t))


def _case(T, hq, hkv, dh, rot, norm, seed=0, far=977, std=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = (std * torch.randn(T, (hq + 2 * hkv) * dh, generator=g)).to(torch.bfloat16).cuda()
    q, k, v = (x.view(T, -1, dh) for x in qkv.split([hq * dh, hkv * dh, hkv * dh], 1))
    w = [(1 + 0.3 * torch.randn(dh, generator=g)).to(torch.bfloat16).cuda() if norm else None for _ in range(2)]
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
    return qkv, q, k, v, w, pos, pa.rope_table(far, rot, device="cuda")


def _check(got, x, w, offset, eps, pos, table, interleaved):
    want, size = ref.norm_rope(_f64(x), None if w is None else _f64(w), offset, eps, pos.cpu().numpy(),
                               table.cpu().numpy(), interleaved)
    tol = np.abs(want) * 2.0 ** -8 + size * 24 * 2.0 ** -24 + 1e-38
    live = pos.cpu().numpy() >= 0
    err = np.abs(_f64(got) - want)[live]
    assert (err <= tol[live]).all(), float((err / tol[live]).max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,dh,rot,norm", [
    (1, 8, 2, 128, 128, True), (3, 1, 1, 128, 64, True), (64, 8, 2, 128, 128, False), (77, 7, 1, 128, 16, True),
    (130, 16, 2, 256, 64, True), (33, 8, 2, 256, 256, True), (19, 3, 1, 512, 512, True), (20, 4, 2, 512, 48, False),
    (3001, 32, 8, 128, 128, True), (5, 128, 1, 128, 112, True)])
def test_matches_formula(T, hq, hkv, dh, rot, norm, interleaved):
    _, q, k, _, w, pos, table = _case(T, hq, hkv, dh, rot, norm)
    qo, ko = pa.qk_norm_rope(q, k, pos, table, q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=interleaved)
    assert pa.check_errors() == (pa.PA_OK, -1)
    _check(qo, q, w[0], 0.0, 1e-5, pos, table, interleaved)
    _check(ko, k, w[1], 0.0, 1e-5, pos, table, interleaved)


def test_one_norm_only_weight_offset_and_in_place():
    qkv, q, k, v, w, pos, table = _case(50, 8, 2, 128, 128, True, seed=4)
    before = qkv.clone()
    q0, k0 = (before[:, a:b].reshape(50, -1, 128) for a, b in ((0, 1024), (1024, 1280)))
    pa.qk_norm_rope(q, k, pos, table, q, k, q_weight=None, k_weight=w[1], weight_offset=1.0)
    assert pa.check_errors() == (pa.PA_OK, -1)
    _check(q, q0, None, 1.0, 1e-6, pos, table, False)
    _check(k, k0, w[1], 1.0, 1e-6, pos, table, False)
    assert torch.equal(qkv[:, 1280:].view(torch.int16), before[:, 1280:].view(torch.int16))


@pytest.mark.parametrize("std,eps", [(1e30, 1e-6), (1e-25, 0.0), (1e-25, 1e-6), (1e19, 0.0), (3e37, 1.0), (1e-30, 2.0)])
def test_rows_whose_squares_leave_the_range(std, eps):
    _, q, k, _, w, pos, table = _case(40, 4, 2, 128, 128, True, seed=5, std=std)
    qo, ko = pa.qk_norm_rope(q, k, pos, table, q_weight=w[0], k_weight=w[1], eps=eps)
    _check(qo, q, w[0], 0.0, eps, pos, table, False)
    _check(ko, k, w[1], 0.0, eps, pos, table, False)


def test_zero_rows_and_nonfinite_rows_stay_in_their_place():
    _, q, k, _, w, pos, table = _case(9, 4, 2, 128, 128, True, seed=6)
    q = q.clone()
    q[2] = 0
    q[3, 1, 5] = float("nan")
    q[4, 2, 100] = float("inf")
    qo, _ = pa.qk_norm_rope(q, k, pos, table, q_weight=w[0], k_weight=w[1])
    assert bool((qo[2] == 0).all())
    assert bool(qo[3, 1].isnan().all()) and not bool(qo[3, 0].isnan().any())
    assert not bool(qo[4, [0, 1, 3]].isnan().any()) and not bool(qo[5:].isnan().any())


def test_padding_rows_untouched_and_far_positions():
    _, q, k, _, w, pos, table = _case(12, 8, 2, 128, 128, True, seed=7)
    pos = pos.clone()
    pos[[1, 11]] = -1
    pos[0], pos[2] = 0, 976
    qo, ko = (torch.full(x.shape, 0, dtype=torch.int16, device="cuda").add_(FILL).view(torch.bfloat16) for x in (q, k))
    pa.qk_norm_rope(q, k, pos, table, qo, ko, w[0], w[1])
    assert pa.check_errors() == (pa.PA_OK, -1)
    assert (bits(qo[[1, 11]]) == FILL).all() and (bits(ko[[1, 11]]) == FILL).all()
    _check(qo, q, w[0], 0.0, 1e-6, pos, table, False)
    pos[4] = 977
    pa.qk_norm_rope(q, k, pos, table, qo, ko, w[0], w[1])
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 4)
    assert bool(qo[4].isnan().all()) and bool(ko[4].isnan().all()) and not bool(qo[5].isnan().any())


@pytest.mark.parametrize("layout", ["separate", "interleaved", "head_major"])
@pytest.mark.parametrize("T,hq,hkv,dh", [(1, 8, 2, 128), (61, 7, 1, 256), (40, 8, 2, 512), (700, 16, 4, 128)])
def test_with_cache_write_equals_the_two_calls(T, hq, hkv, dh, layout):
    _, q, k, v, w, pos, table = _case(T, hq, hkv, dh, 64, True, seed=8)
    blocks = T // 16 + 3
    if layout == "head_major":
        make = lambda: torch.zeros(2, blocks, hkv, 16, dh, dtype=torch.bfloat16, device="cuda").transpose(2, 3)
    elif layout == "interleaved":
        make = lambda: torch.zeros(blocks, 2, 16, hkv, dh, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    else:
        make = lambda: torch.zeros(2, blocks, 16, hkv, dh, dtype=torch.bfloat16, device="cuda")
    slots = torch.randperm(blocks * 16, generator=torch.Generator().manual_seed(1))[:T].cuda()
    if T > 5:
        slots[3], pos = -1, pos.clone()
        pos[5] = -1                       # padding: nothing written
    a, b = make(), make()
    qa = pa.qk_norm_rope_and_cache(q, k, v, pos, table, a[0], a[1], slots, q_weight=w[0], k_weight=w[1])
    qb, kb = pa.qk_norm_rope(q, k, pos, table, q_weight=w[0], k_weight=w[1])
    two = slots.clone()
    two[pos < 0] = -1
    pa.reshape_and_cache(kb, v, b[0], b[1], two)
    assert pa.check_errors() == (pa.PA_OK, -1)
    live = pos >= 0
    assert torch.equal(qa[live].view(torch.int16), qb[live].view(torch.int16))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_cache_write_with_bad_slot_and_bad_position():
    _, q, k, v, w, pos, table = _case(20, 8, 2, 128, 128, True, seed=9)
    pool = torch.zeros(2, 4, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(20, device="cuda")
    slots[7] = 64
    pa.qk_norm_rope_and_cache(q, k, v, pos, table, pool[0], pool[1], slots, q_weight=w[0], k_weight=w[1])
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 7)
    assert not bool(pool[:, 0, 7].any()) and bool(pool[:, 0, 8].any())
    pos = pos.clone()
    pos[9] = 5000
    pool.zero_()
    slots[7] = 7
    pa.qk_norm_rope_and_cache(q, k, v, pos, table, pool[0], pool[1], slots, q_weight=w[0], k_weight=w[1])
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 9)
    assert not bool(pool[:, 0, 9].any()) and bool(pool[:, 0, 8].any())


def test_pool_past_two_to_the_31_elements():
    T, hkv, dh, blocks = 4, 8, 512, 33000
    _, q, k, v, w, pos, table = _case(T, 8, hkv, dh, 128, True, seed=10)
    pool = torch.zeros(2, blocks, 16, hkv, dh, dtype=torch.bfloat16, device="cuda")
    assert pool[0].numel() > 2**31
    slots = torch.tensor([blocks * 16 - 1, 0, (blocks - 1) * 16, 5], device="cuda")
    pa.qk_norm_rope_and_cache(q, k, v, pos, table, pool[0], pool[1], slots, q_weight=w[0], k_weight=w[1])
    _, kb = pa.qk_norm_rope(q, k, pos, table, q_weight=w[0], k_weight=w[1])
    assert pa.check_errors() == (pa.PA_OK, -1)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(pool[0, s // 16, s % 16].view(torch.int16), kb[i].view(torch.int16))
        assert torch.equal(pool[1, s // 16, s % 16].view(torch.int16), v[i].view(torch.int16))
