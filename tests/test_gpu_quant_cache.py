"""The 4-bit cache: pa_reshape_and_cache_quant byte for byte against a plain
64-bit quantiser (ties to even, saturation, zero, NaN and infinite blocks), and
pa_dequantize_kv value for value (every value is exact in BF16)."""
import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import step_reference as ref
from tests.helpers import bits, bits_to_f64

pytestmark = pytest.mark.gpu


def _f64(t):
    return bits_to_f64(bits(t))


def _pool(blocks, hkv, dh, layout, fill=0xA5):
    rec = pa.quant_record_bytes(dh)
    if layout == "interleaved":
        p = torch.full((blocks, 2, hkv, rec), fill, dtype=torch.uint8, device="cuda")
        return p[:, 0], p[:, 1]
    if layout == "padded":
        p = torch.full((2, blocks, hkv, rec + 48), fill, dtype=torch.uint8, device="cuda")
        return p[0, ..., :rec], p[1, ..., :rec]
    p = torch.full((2, blocks, hkv, rec), fill, dtype=torch.uint8, device="cuda")
    return p[0], p[1]


def _expect(before, x, slots, which, dh, scale):
    """The pool's bytes after the write, from `before`."""
    after = before.copy()
    codes, sc = ref.quantise(x, scale)
    data = codes[..., 0::2] | codes[..., 1::2] << 4
    for i, s in enumerate(slots):
        if s < 0:
            continue
        rec = after[s // 16]
        body, tail = rec[:, :8 * dh], rec[:, 8 * dh:]
        if which == "k":
            body.reshape(-1, 16, dh // 2)[:, s % 16] = data[i]
            tail.reshape(-1, 16, dh // 16)[:, s % 16] = sc[i]
        else:
            body.reshape(-1, dh // 2, 16)[:, :, s % 16] = data[i]
            tail.reshape(-1, dh // 16, 16)[:, :, s % 16] = sc[i]
        rec[:, :8 * dh], rec[:, 8 * dh:] = body, tail
    return after


def _tokens(T, hkv, dh, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(T, 2 * hkv * dh, generator=g)
    if kind == "ties":
        # small whole multiples of a power of two: the codes' and scales' ties are common
        kv = torch.randint(-48, 49, kv.shape, generator=g) * 0.125
    elif kind == "wide":
        kv = kv * torch.exp2(torch.randint(-18, 18, (T, 1), generator=g).float())
    kv = kv.to(torch.bfloat16).cuda()
    return kv[:, :hkv * dh].view(T, hkv, dh), kv[:, hkv * dh:].view(T, hkv, dh)


def _write_and_check(k, v, slots, blocks, layout="separate", k_scale=1.0, v_scale=1.0):
    hkv, dh = k.shape[1:]
    kp, vp = _pool(blocks, hkv, dh, layout)
    cache = pa.QuantCache(kp, vp, dh, k_scale, v_scale)
    before = [p.cpu().numpy().copy() for p in (kp, vp)]
    pa.reshape_and_cache_quant(k, v, cache, slots)
    for p, b, x, which, s in ((kp, before[0], k, "k", k_scale), (vp, before[1], v, "v", v_scale)):
        want = _expect(b, _f64(x), slots.tolist(), which, dh, s)
        got = p.cpu().numpy()
        assert np.array_equal(got, want), (which, np.argwhere(got != want)[:5])
    return cache


@pytest.mark.parametrize("kind", ["normal", "ties", "wide"])
@pytest.mark.parametrize("T,hkv,dh,layout", [(1, 1, 128, "separate"), (17, 2, 128, "interleaved"),
                                             (250, 8, 128, "padded"), (33, 2, 256, "separate"),
                                             (19, 1, 512, "interleaved")])
def test_write_matches_quantiser_byte_for_byte(T, hkv, dh, layout, kind):
    k, v = _tokens(T, hkv, dh, T + dh, kind)
    blocks = T // 16 + 3
    slots = torch.randperm(blocks * 16, generator=torch.Generator().manual_seed(T))[:T].cuda()
    if T > 4:
        slots[2] = -1
    _write_and_check(k, v, slots, blocks, layout, 0.25, 2.0)
    assert pa.check_errors() == (pa.PA_OK, -1)


@pytest.mark.parametrize("start", [0, 3, 8])
def test_consecutive_slots_as_in_a_prompt(start):
    k, v = _tokens(100, 2, 128, start)
    _write_and_check(k, v, torch.arange(start, start + 100, device="cuda"), 9)


@pytest.mark.parametrize("scale", [2.0 ** -32, 1.0, 2.0 ** 32])
def test_saturation_zero_and_nonfinite_blocks(scale):
    k, v = _tokens(8, 1, 128, 3)
    k, v = k.clone(), v.clone()
    k[0, 0, :16] = 0
    k[1, 0, 16:32] = float("nan")
    k[2, 0, 40] = float("inf")
    k[3, 0, 50] = -float("inf")
    k[4, 0, 64:80] = 3e38            # far above the largest scale
    k[4, 0, 65] = -3e38
    k[5, 0, :16] = 1e-39             # subnormal
    k[6, 0, 5] = 2.0 ** -120
    k[7, 0, 16:32] = -0.0
    v[0, 0, 3] = float("nan")
    cache = _write_and_check(k, v, torch.arange(8, device="cuda"), 1, k_scale=scale, v_scale=scale)
    vals = ref.pool_values(cache.k_pool.cpu().numpy(), "k", 128, scale)[0]
    assert np.isnan(vals[1, 0, 16:32]).all() and np.isnan(vals[2, 0, 32:48]).all() and np.isnan(vals[3, 0, 48:64]).all()
    assert np.isfinite(vals[2, 0, :32]).all() and np.isfinite(vals[4, 0]).all()
    if scale == 1.0:
        assert vals[4, 0, 64] == 2688 and vals[4, 0, 65] == -2688


def test_bad_slot_is_reported_and_not_written():
    k, v = _tokens(20, 2, 128, 5)
    kp, vp = _pool(2, 2, 128, "separate")
    slots = torch.arange(20, device="cuda")
    slots[11] = 32
    pa.reshape_and_cache_quant(k, v, pa.QuantCache(kp, vp, 128), slots)
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 11)
    want = slots.clone()
    want[11] = -1
    b = np.full(tuple(kp.shape), 0xA5, np.uint8)
    assert np.array_equal(kp.cpu().numpy(), _expect(b, _f64(k), want.tolist(), "k", 128, 1.0))


def _random_cache(blocks, hkv, dh, layout, seed, k_scale=0.5, v_scale=4.0):
    rec = pa.quant_record_bytes(dh)
    g = torch.Generator().manual_seed(seed)
    kp, vp = _pool(blocks, hkv, dh, layout)
    for p in (kp, vp):
        x = torch.randint(0, 256, (blocks, hkv, rec), generator=g, dtype=torch.uint8)
        x[..., 8 * dh:] %= 0x7F       # every scale value there is
        p.copy_(x)
    return pa.QuantCache(kp, vp, dh, k_scale, v_scale)


def _table(lens, blocks, cols, seed):
    rng = np.random.default_rng(seed)
    perm, at = rng.permutation(blocks), 0
    t = np.full((len(lens), cols), 2**31 - 1, np.int32)
    for b, n in enumerate(lens):
        m = -(-n // 16)
        t[b, :m] = perm[at:at + m]
        at += m
    return torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def _buffers(cap, hkv, dh, n, cols):
    out = torch.full((2, cap, 16, hkv, dh), 0, dtype=torch.int16, device="cuda").add_(0x7FC3).view(torch.bfloat16)
    return out[0], out[1], torch.full((n, cols), 77, dtype=torch.int32, device="cuda"), \
        torch.full((n + 1,), 77, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens,hkv,dh,layout", [
    ([1], 1, 128, "separate"), ([37, 16, 50, 1, 0, 29, 300], 2, 128, "interleaved"), ([100, 15], 8, 128, "padded"),
    ([33, 0, 64], 2, 256, "separate"), ([90, 5], 2, 512, "interleaved"), ([0, 0], 2, 128, "separate"),
    ([17] * 700, 1, 128, "separate")])
def test_read_back_is_exact(lens, hkv, dh, layout):
    total = sum(-(-n // 16) for n in lens)
    cols = max(-(-n // 16) for n in lens) + 2
    cache = _random_cache(total + 5, hkv, dh, layout, dh + len(lens))
    bt, sl = _table(lens, total + 5, cols, 3)
    ko, vo, ct, co = _buffers(total + 2, hkv, dh, len(lens), cols)
    pa.dequantize_kv(cache, bt, sl, ko, vo, ct, co)
    assert pa.check_errors() == (pa.PA_OK, -1)
    ids = np.concatenate([bt[b, :-(-n // 16)].cpu().numpy() for b, n in enumerate(lens)]).astype(int)
    for got, pool, which, s in ((ko, cache.k_pool, "k", 0.5), (vo, cache.v_pool, "v", 4.0)):
        want = ref.pool_values(pool.cpu().numpy(), which, dh, s)[ids]
        assert np.array_equal(_f64(got[:total]), want)
        assert (bits(got[total:]) == 0x7FC3).all()
    off = np.concatenate([[0], np.cumsum([-(-n // 16) for n in lens])])
    assert np.array_equal(co.cpu().numpy(), off)
    want = np.full((len(lens), cols), -1)
    for b in range(len(lens)):
        want[b, :off[b + 1] - off[b]] = np.arange(off[b], off[b + 1])
    assert np.array_equal(ct.cpu().numpy(), want)


def test_read_back_errors():
    lens = [40, 20, 33]
    cache = _random_cache(16, 2, 128, "separate", 1)
    bt, sl = _table(lens, 16, 4, 5)
    ref_out = _buffers(8, 2, 128, 3, 4)
    pa.dequantize_kv(cache, bt, sl, *ref_out)
    # a bad block id: its page is NaN, the others are as before
    bad = bt.clone()
    bad[1, 1] = 16
    ko, vo, ct, co = _buffers(8, 2, 128, 3, 4)
    pa.dequantize_kv(cache, bad, sl, ko, vo, ct, co)
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 1)
    assert bool(ko[4].isnan().all()) and bool(vo[4].isnan().all())
    keep = [0, 1, 2, 3, 5, 6, 7]
    assert torch.equal(ko[keep].view(torch.int16), ref_out[0][keep].view(torch.int16))
    # a bad length selects nothing
    ko, vo, ct, co = _buffers(8, 2, 128, 3, 4)
    pa.dequantize_kv(cache, bt, torch.tensor([40, 65, 33], dtype=torch.int32, device="cuda"), ko, vo, ct, co)
    assert pa.check_errors() == (pa.PA_ERR_BAD_METADATA, 1)
    assert co.tolist() == [0, 3, 3, 6] and ct[1].tolist() == [-1] * 4
    # too little room: offsets only
    ko, vo, ct, co = _buffers(7, 2, 128, 3, 4)
    pa.dequantize_kv(cache, bt, sl, ko, vo, ct, co)
    assert pa.check_errors() == (pa.PA_ERR_WORKSPACE, 8)
    assert co.tolist() == [0, 3, 5, 8] and bool((ct == 77).all()) and (bits(ko) == 0x7FC3).all()


def test_pool_past_two_to_the_32_bytes():
    hkv, dh = 8, 512
    blocks = 2**32 // (hkv * 9 * dh) + 3
    kp = torch.zeros(blocks, hkv, 9 * dh, dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    cache = pa.QuantCache(kp, vp, dh)
    k, v = _tokens(3, hkv, dh, 8)
    slots = torch.tensor([blocks * 16 - 1, 0, (blocks - 1) * 16 + 4], device="cuda")
    pa.reshape_and_cache_quant(k, v, cache, slots)
    bt = torch.tensor([[blocks - 1, 0]], dtype=torch.int32, device="cuda")
    ko, vo, ct, co = _buffers(2, hkv, dh, 1, 2)
    pa.dequantize_kv(cache, bt, torch.tensor([17], dtype=torch.int32, device="cuda"), ko, vo, ct, co)
    assert pa.check_errors() == (pa.PA_OK, -1)
    for out, x in ((ko, k), (vo, v)):
        want = ref.values(*ref.quantise(_f64(x), 1.0), 1.0)
        got = _f64(out)
        assert np.array_equal(got[0, 15], want[0]) and np.array_equal(got[1, 0], want[1]) and np.array_equal(got[0, 4], want[2])
