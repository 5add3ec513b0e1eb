"""The C-ABI checks of the step metadata, the norm and rotation, and the 4-bit
cache without a GPU: bad arguments are refused on the host before any CUDA
call, sound ones get as far as CUDA."""
import ctypes

import pytest
import torch

from paged_kv_cache_178_gb300 import build as pa_build
from paged_kv_cache_178_gb300 import pagedattn as pa

INVALID, UNSUPPORTED, OK, WORKSPACE = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_OK, pa.PA_ERR_WORKSPACE

# Aligned addresses 64 MB apart, never dereferenced.
NAMES = ("ctx", "new", "bt", "free", "cin", "cout", "slots", "pos", "sl", "qsl", "q", "k", "v", "cos", "qw", "kw", "qo",
         "ko", "pk", "pv", "out", "lse", "ws", "kout", "vout", "ct", "co")
AT = {n: (i + 1) << 26 for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


def _reaches_cuda(rc):
    """A sound call: without a GPU it fails in CUDA; with one it is not issued."""
    return rc == pa.PA_ERR_CUDA


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real ones")


def _meta(lib, **kw):
    a = dict(AT, n=4, cols=448, nfree=1000, blocks=2048, tokens=64)
    a.update(kw)
    return lib.pa_build_step_metadata(a["ctx"], a["new"], a["n"], a["bt"], a["cols"], a["free"], a["nfree"], a["cin"],
                                      a["cout"], a["blocks"], a["slots"], a["pos"], a["tokens"], a["sl"], a["qsl"], None)


def test_step_metadata_refusals(lib):
    for kw in (dict(n=-1), dict(cols=0), dict(nfree=-1), dict(blocks=0), dict(blocks=2**31 + 1), dict(tokens=-1),
               dict(tokens=2**31), dict(ctx=0), dict(new=0), dict(bt=0), dict(cout=0), dict(sl=0), dict(qsl=0),
               dict(free=0), dict(slots=0), dict(pos=0), dict(ctx=AT["ctx"] + 2), dict(slots=AT["slots"] + 4),
               dict(qsl=AT["qsl"] + 1)):
        assert _meta(lib, **kw) == INVALID, kw
    for kw in (dict(n=8193), dict(cols=(2**31 - 1) // 16 + 1)):
        assert _meta(lib, **kw) == UNSUPPORTED, kw
    assert _meta(lib, n=0, ctx=0, bt=0) == OK
    # outputs that share bytes with an input or another output
    for kw in (dict(bt=AT["ctx"]), dict(sl=AT["new"]), dict(sl=AT["ctx"] + 4), dict(qsl=AT["new"]),
               dict(slots=AT["free"] + 3992), dict(pos=AT["sl"]), dict(cout=AT["cin"], sl=AT["cin"]),
               dict(cout=AT["free"]), dict(pos=AT["slots"] + 8 * 63), dict(qsl=AT["sl"] + 12)):
        assert _meta(lib, **kw) == INVALID, kw


@needs_no_gpu
def test_step_metadata_sound_calls(lib):
    for kw in (dict(), dict(sl=AT["ctx"], cout=AT["cin"]), dict(cin=0), dict(tokens=0, slots=0, pos=0),
               dict(nfree=0, free=0), dict(n=8192), dict(pos=AT["slots"] + 8 * 64)):
        assert _reaches_cuda(_meta(lib, **kw)), kw


def _rope(lib, cache=None, **kw):
    a = dict(AT, hq=8, hkv=2, dh=128, n=4, maxp=8192, rot=128, inter=0, off=0.0, eps=1e-6, qs=1024, ks=256, vs=256,
             qos=1024, kos=256)
    a.update(kw)
    f = ctypes.c_float
    if cache is None:
        return lib.pa_qk_norm_rope(a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["hkv"], a["dh"], a["n"], a["pos"], a["cos"],
                                   a["maxp"], a["rot"], a["inter"], a["qw"], a["kw"], f(a["off"]), f(a["eps"]), a["qo"],
                                   a["qos"], a["ko"], a["kos"], None)
    return lib.pa_qk_norm_rope_and_cache(a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["v"], a["vs"], a["n"], a["pos"],
                                         a["cos"], a["maxp"], a["rot"], a["inter"], a["qw"], a["kw"], f(a["off"]),
                                         f(a["eps"]), a["qo"], a["qos"], ctypes.byref(cache), a["slots"], None)


def _bf16_cache(**kw):
    c = dict(k=AT["pk"], v=AT["pv"], num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128, kv_tile=0,
             block_stride=16 * 256, token_stride=256, head_stride=128)
    c.update(kw)
    return pa.PaKvCache(**c)


FUSED = dict(qs=1536, ks=1536, vs=1536, k=AT["q"] + 2048, v=AT["q"] + 2560)  # slices of one [T, 12, 128] projection


def test_norm_and_rotation_refusals(lib):
    c = _bf16_cache()
    for cache in (None, c):
        for kw in (dict(n=-1), dict(n=2**31), dict(maxp=0), dict(hq=0), dict(eps=-1.0), dict(eps=float("inf")),
                   dict(eps=float("nan")), dict(off=float("nan")), dict(off=float("inf")), dict(q=0), dict(k=0), dict(qo=0),
                   dict(pos=0), dict(cos=0), dict(q=AT["q"] + 2), dict(qs=1020), dict(qs=1000), dict(ks=252),
                   dict(qos=1016), dict(cos=AT["cos"] + 4), dict(qw=AT["qw"] + 2), dict(pos=AT["pos"] + 1)):
            assert _rope(lib, cache, **kw) == INVALID, kw
        for kw in (dict(rot=8), dict(rot=0), dict(rot=24), dict(rot=144)):
            assert _rope(lib, cache, **kw) == UNSUPPORTED, kw
        assert _rope(lib, cache, n=0, q=0) == OK
        # outputs over other arguments; in place with another stride or start
        for kw in (dict(qo=AT["q"], qos=1032), dict(qo=AT["q"] + 16), dict(qo=AT["k"]), dict(qo=AT["cos"] + 16),
                   dict(qo=AT["qw"]), dict(qo=AT["pos"]), dict(FUSED, qo=AT["q"] + 1024, qos=1536)):
            assert _rope(lib, cache, **kw) == INVALID, kw
    for kw in (dict(hkv=0), dict(ko=0), dict(ko=AT["qo"]), dict(ko=AT["q"]), dict(ko=AT["k"] + 16), dict(kos=248)):
        assert _rope(lib, **kw) == INVALID, kw
    assert _rope(lib, dh=64) == UNSUPPORTED
    for kw in (dict(v=0), dict(vs=200), dict(slots=0), dict(slots=AT["slots"] + 4), dict(qo=AT["v"]), dict(qo=AT["pk"]),
               dict(k=AT["pv"] + 4096), dict(slots=AT["pk"]), dict(v=AT["pk"])):
        assert _rope(lib, c, **kw) == INVALID, kw
    assert _rope(lib, _bf16_cache(head_dim=64)) == UNSUPPORTED
    assert _rope(lib, _bf16_cache(k=0)) == INVALID


@needs_no_gpu
def test_norm_and_rotation_sound_calls(lib):
    fused_in_place = dict(FUSED, qo=AT["q"], qos=1536)
    for kw in (dict(), dict(qw=0, kw=0), dict(rot=16, inter=1), dict(qo=AT["q"]), fused_in_place, dict(eps=0.0)):
        assert _reaches_cuda(_rope(lib, _bf16_cache(), **kw)), kw
        assert _reaches_cuda(_rope(lib, **kw)), kw
    assert _reaches_cuda(_rope(lib, **dict(fused_in_place, ko=FUSED["k"], kos=1536)))


def _quant(**kw):
    c = dict(k=AT["pk"], v=AT["pv"], num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128, reserved=0,
             block_stride=2 * 1152, head_stride=1152, k_scale=1.0, v_scale=0.25)
    c.update(kw)
    return pa.PaQuantCache(**c)


BAD_POOLS = [(dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k=AT["pk"] + 8), INVALID), (dict(num_blocks=0), INVALID),
             (dict(num_blocks=2**31 + 1), INVALID), (dict(num_kv_heads=0), INVALID), (dict(reserved=1), INVALID),
             (dict(block_size=32), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED), (dict(block_stride=0), INVALID),
             (dict(block_stride=2 * 1152 + 8), INVALID), (dict(head_stride=1136), INVALID),
             (dict(block_stride=2**32), UNSUPPORTED), (dict(head_stride=2**32), UNSUPPORTED), (dict(k_scale=0.0), INVALID),
             (dict(k_scale=3.0), INVALID), (dict(v_scale=-1.0), INVALID), (dict(v_scale=float("nan")), INVALID),
             (dict(v_scale=float("inf")), INVALID), (dict(k_scale=2.0**-33), INVALID), (dict(k_scale=2.0**33), INVALID)]


def _write(lib, cache, **kw):
    a = dict(AT, ks=256, vs=256, n=4)
    a.update(kw)
    return lib.pa_reshape_and_cache_quant(a["k"], a["ks"], a["v"], a["vs"], a["n"], ctypes.byref(cache), a["slots"], None)


def _read(lib, cache, **kw):
    a = dict(AT, cols=8, n=4, cap=32)
    a.update(kw)
    return lib.pa_dequantize_kv(ctypes.byref(cache), a["bt"], a["cols"], a["sl"], a["n"], a["kout"], a["vout"], a["cap"],
                                a["ct"], a["co"], None)


def _attend(lib, cache, **kw):
    a = dict(AT, tq=4, qs=1024, hq=8, cols=448, n=4, mq=1, ms=7168, pages=0, scale=0.088, ws_len=None)
    a.update(kw)
    if a["ws_len"] is None:
        a["ws_len"] = pa.quant_workspace_size(a["n"], a["hq"], cache.num_kv_heads, cache.head_dim, a["mq"], a["ms"],
                                              a["pages"])
    return lib.pa_paged_attention_quant(a["q"], a["tq"], a["qs"], a["hq"], ctypes.byref(cache), a["bt"], a["cols"], a["sl"],
                                        a["qsl"], a["n"], a["mq"], a["ms"], a["pages"], ctypes.c_float(a["scale"]), a["out"],
                                        a["lse"], a["ws"], a["ws_len"], None)


@pytest.mark.parametrize("kw,status", BAD_POOLS)
def test_bad_pools_are_refused_by_every_call(lib, kw, status):
    c = _quant(**kw)
    assert _write(lib, c) == status and _read(lib, c) == status
    assert _attend(lib, c, ws_len=1 << 20) == status


def test_write_and_read_back_refusals(lib):
    c = _quant()
    for kw in (dict(n=-1), dict(k=0), dict(v=0), dict(slots=0), dict(ks=248), dict(ks=252), dict(k=AT["k"] + 8),
               dict(slots=AT["slots"] + 4), dict(k=AT["pk"]), dict(v=AT["pv"] + 64 * 2304 - 16), dict(slots=AT["pv"])):
        assert _write(lib, c, **kw) == INVALID, kw
    assert _write(lib, c, n=0, k=0) == OK
    for kw in (dict(n=-1), dict(cols=0), dict(cap=-1), dict(bt=0), dict(sl=0), dict(ct=0), dict(co=0), dict(kout=0),
               dict(vout=AT["vout"] + 8), dict(bt=AT["bt"] + 2), dict(kout=AT["pk"]), dict(vout=AT["kout"]),
               dict(ct=AT["bt"]), dict(co=AT["ct"] + 124), dict(co=AT["sl"])):
        assert _read(lib, c, **kw) == INVALID, kw
    assert _read(lib, c, n=8193) == UNSUPPORTED
    assert _read(lib, c, n=8192, cols=2**18) == UNSUPPORTED
    assert _read(lib, c, n=0, bt=0) == OK


def test_attention_refusals(lib):
    c = _quant()
    need = pa.quant_workspace_size(4, 8, 2, 128, 1, 7168)
    for kw in (dict(tq=-1), dict(tq=2**31), dict(n=-1), dict(mq=-1), dict(ms=-1), dict(cols=-1), dict(cols=0), dict(pages=-1),
               dict(hq=0), dict(q=0), dict(out=0), dict(bt=0), dict(sl=0), dict(qsl=0), dict(q=AT["q"] + 2), dict(qs=1000),
               dict(qs=1028), dict(out=AT["out"] + 8), dict(lse=AT["lse"] + 2), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=AT["ws"] + 16), dict(out=AT["q"]),
               dict(out=AT["pk"]), dict(lse=AT["out"]), dict(ws=AT["q"]), dict(ws=AT["pv"]), dict(out=AT["ws"] + 256),
               dict(lse=AT["sl"]), dict(out=AT["bt"] + 4 * 448 * 4 - 16)):
        assert _attend(lib, c, **dict(dict(ws_len=need), **kw)) == INVALID, kw
    assert _attend(lib, c, hq=7) == UNSUPPORTED
    assert _attend(lib, c, hq=2 * 129) == UNSUPPORTED
    assert _attend(lib, c, n=2049, ms=16) == UNSUPPORTED
    assert _attend(lib, c, n=2048, ms=16 * (2**17 + 1), cols=2**17 + 1) == UNSUPPORTED
    for kw in (dict(ws=0), dict(ws_len=0), dict(ws_len=need - 1)):
        assert _attend(lib, c, **kw) == WORKSPACE, kw
    for kw in (dict(n=0), dict(tq=0), dict(mq=0)):
        assert _attend(lib, c, **dict(kw, q=0, ws=0)) == OK, kw


@needs_no_gpu
def test_4bit_sound_calls(lib):
    c = _quant()
    both = _quant(v=AT["pk"] + 2304, block_stride=2 * 2304)  # one interleaved pool
    for cache in (c, both, _quant(k_scale=2.0**-32, v_scale=2.0**32)):
        assert _reaches_cuda(_write(lib, cache)) and _reaches_cuda(_read(lib, cache))
        assert _reaches_cuda(_attend(lib, cache, lse=0)) and _reaches_cuda(_attend(lib, cache))
    assert _reaches_cuda(_read(lib, c, cap=0, kout=0, vout=0))
    assert _reaches_cuda(_attend(lib, c, mq=100, tq=400, ms=100))


def test_workspace_sizes():
    size = pa.quant_workspace_size
    for bad in ((4, 7, 2, 128, 1, 100), (4, 8, 2, 64, 1, 100), (-1, 8, 2, 128, 1, 100), (4, 8, 2, 128, 1, 100, -1),
                (2049, 8, 2, 128, 1, 100), (4, 8, 0, 128, 1, 100)):
        assert size(*bad) == 0, bad
    # one fp32 record of rows x (Dh + 2) per 512 keys and KV head, at least
    n = size(4, 8, 2, 128, 1, 7168)
    assert n >= 4 * 2 * 14 * 4 * 130 * 4 and n % 4 == 0
    # a bound of the pages shrinks both kinds
    assert size(64, 8, 2, 128, 1, 7168, 500) < size(64, 8, 2, 128, 1, 7168)
    assert size(64, 8, 2, 128, 50, 7168, 500) < size(64, 8, 2, 128, 50, 7168)
    assert size(64, 8, 2, 128, 1, 7168, 10**9) == size(64, 8, 2, 128, 1, 7168)


def test_binding_refuses_host_tensors():
    i32, bf = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 9 * 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pa.QuantCache(pool, pool.clone(), 128)
    with pytest.raises(ValueError):
        pa.build_step_metadata(i32, i32, i32.view(1, 4), i32, 4, i32.long(), i32, i32, i32, i32)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(bf, bf, i32, torch.zeros(8, 128), bf, bf)
    assert pa.quant_record_bytes(256) == 2304


def test_rope_table_values():
    t = pa.rope_table(70, 32, 10000.0)
    assert t.shape == (70, 32) and t.dtype == torch.float32
    p = torch.arange(70, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)
    # one rounding of values up to 1, and the 64-bit angle's own
    assert (t[:, :16].double() - p.cos()).abs().max() <= 2.0 ** -25 + 2.0 ** -40
    assert (t[:, 16:].double() - p.sin()).abs().max() <= 2.0 ** -25 + 2.0 ** -40
