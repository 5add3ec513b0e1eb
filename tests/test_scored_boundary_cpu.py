"""The C-ABI checks of pa_paged_attention_scored without a GPU: bad arguments
are refused on the host before any CUDA call, sound ones get as far as CUDA."""
import ctypes
import math

import pytest
import torch

from paged_kv_cache_178_gb300 import build as pa_build
from paged_kv_cache_178_gb300 import pagedattn as pa

INVALID, UNSUPPORTED, OK, WORKSPACE = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_OK, pa.PA_ERR_WORKSPACE

# Aligned addresses 1 GB apart, never dereferenced.
NAMES = ("q", "k", "v", "bt", "sl", "qsl", "slopes", "prefix", "first", "out", "lse", "ws")
AT = {n: (i + 1) << 30 for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real ones")


def _call(lib, cache=None, rules=None, **kw):
    c = dict(k=AT["k"], v=AT["v"], num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128, kv_tile=0,
             block_stride=16 * 256, token_stride=256, head_stride=128)
    c.update(cache or {})
    a = dict(q=AT["q"], t=20, stride=None, hq=8, bt=AT["bt"], cols=40, sl=AT["sl"], qsl=AT["qsl"], seqs=4, mq=5, ms=600,
             scale=0.1, out=AT["out"], lse=AT["lse"], ws=AT["ws"], bytes=1 << 29)
    a.update(kw)
    r = None
    if rules is not None:
        r = ctypes.byref(pa.PaScoreRules(rules.get("cap", 0.0), rules.get("window", 0), rules.get("slopes", 0),
                                         rules.get("prefix", 0), rules.get("first", 0)))
    stride = a["hq"] * c["head_dim"] if a["stride"] is None else a["stride"]
    return lib.pa_paged_attention_scored(a["q"], a["t"], stride, a["hq"], ctypes.byref(pa.PaKvCache(**c)), a["bt"],
                                         a["cols"], a["sl"], a["qsl"], a["seqs"], a["mq"], a["ms"],
                                         ctypes.c_float(a["scale"]), r, a["out"], a["lse"], a["ws"], a["bytes"], None)


def _size(lib, seqs=4, hq=8, hkv=2, dh=128, mq=5, ms=600):
    return lib.pa_paged_attention_scored_workspace_size(seqs, hq, hkv, dh, mq, ms)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(out=0), dict(bt=0), dict(sl=0), dict(qsl=0), dict(q=AT["q"] + 8), dict(out=AT["out"] + 2),
    dict(lse=AT["lse"] + 2), dict(bt=AT["bt"] + 1), dict(sl=AT["sl"] + 2), dict(qsl=AT["qsl"] + 3), dict(t=-1), dict(seqs=-1),
    dict(mq=-1), dict(ms=-1), dict(cols=-1), dict(cols=0), dict(hq=0), dict(hq=-8), dict(t=2**31), dict(stride=1016),
    dict(stride=1028), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=3e38),
    dict(ws=AT["ws"] + 128), dict(out=AT["q"]), dict(out=AT["k"] + 1024), dict(lse=AT["sl"]), dict(lse=AT["out"] + 1024),
    dict(ws=AT["bt"]), dict(ws=AT["out"]), dict(lse=AT["ws"])], ids=str)
def test_refusals(lib, kw):
    assert _call(lib, **kw) == INVALID


@pytest.mark.parametrize("rules", [
    dict(cap=-1.0), dict(cap=2.0**-21), dict(cap=2.0**21), dict(cap=math.inf), dict(cap=math.nan), dict(window=-1),
    dict(slopes=AT["slopes"] + 2), dict(prefix=AT["prefix"] + 1), dict(first=AT["first"] + 3), dict(slopes=AT["out"]),
    dict(prefix=AT["lse"]), dict(first=AT["ws"])], ids=str)
def test_rule_refusals(lib, rules):
    assert _call(lib, rules=rules) == INVALID


def test_a_scale_too_large_for_a_cap(lib):
    # (the quotient of scale and cap is what the kernels use)
    assert _call(lib, scale=1e35, rules=dict(cap=2.0**-20)) == INVALID


@pytest.mark.parametrize("kw,cache", [
    (dict(hq=7), {}), (dict(hq=258), {}), (dict(), dict(block_size=32)), (dict(), dict(head_dim=64)),
    (dict(seqs=8193, t=8193, mq=1), {}), (dict(mq=2**26), {}), (dict(ms=2**31 - 4095), {}),
    # more row tiles than the schedule holds: 8192 requests of 3 at least
    (dict(seqs=8192, t=8192 * 129, mq=129), {}),
    # more items than 32 bits count: tiles of a long prompt
    (dict(t=2**20, seqs=1, mq=2**20, ms=2**31 - 4096), {})], ids=str)
def test_unsupported(lib, kw, cache):
    if cache.get("head_dim") == 64:
        cache = dict(cache, token_stride=128, head_stride=64, block_stride=16 * 128)
    assert _call(lib, cache=cache, **kw) in (UNSUPPORTED, INVALID if cache else UNSUPPORTED)


def test_cache_refusals(lib):
    for cache in (dict(k=0), dict(v=0), dict(v=AT["v"] + 8), dict(num_blocks=-1), dict(num_kv_heads=0),
                  dict(block_stride=16 * 256 + 4), dict(token_stride=100)):
        assert _call(lib, cache=cache) == INVALID, cache


def test_workspace(lib):
    for mq in (1, 8, 9, 33, 600):
        for dh in (128, 256, 512):
            need = _size(lib, mq=mq, dh=dh)
            assert need > 0
            cache = dict(head_dim=dh, token_stride=2 * dh, head_stride=dh, block_stride=32 * dh)
            for kw in (dict(bytes=need - 1), dict(ws=0), dict(bytes=0)):
                assert _call(lib, cache=cache, mq=mq, **kw) == WORKSPACE, (mq, dh, kw)


def test_workspace_size_of_refused_bounds(lib):
    for kw in (dict(seqs=0), dict(seqs=-1), dict(seqs=8193), dict(hq=0), dict(hkv=0), dict(hq=7), dict(hq=258), dict(dh=64),
               dict(dh=0), dict(mq=0), dict(mq=-1), dict(mq=2**26), dict(ms=-1), dict(ms=2**31 - 4095)):
        assert _size(lib, **kw) == 0, kw


def test_empty_batches(lib):
    for kw in (dict(seqs=0), dict(t=0), dict(mq=0)):
        assert _call(lib, q=0, out=0, lse=0, ws=0, bytes=0, bt=0, sl=0, qsl=0, **kw) == OK
    # (but not with a bad rule or scale)
    assert _call(lib, seqs=0, scale=0.0) == INVALID
    assert _call(lib, seqs=0, rules=dict(window=-1)) == INVALID


def test_more_heads_than_items_count(lib):
    for dh in (128, 256, 512):
        cache = dict(num_kv_heads=20000, head_dim=dh, token_stride=20000 * dh, head_stride=dh, block_stride=16 * 20000 * dh)
        assert _call(lib, cache=cache, hq=20000, seqs=8192, t=8192, mq=1, ms=1024) == UNSUPPORTED


@needs_no_gpu
def test_sound_calls(lib):
    every = dict(cap=50.0, window=1, slopes=AT["slopes"], prefix=AT["prefix"], first=AT["first"])
    for mq in (1, 5, 8, 9, 600):
        for rules in (None, {}, every, dict(cap=2.0**-20), dict(cap=2.0**20, window=2**31 - 1)):
            assert _call(lib, mq=mq, rules=rules) == pa.PA_ERR_CUDA
    assert _call(lib, lse=0) == pa.PA_ERR_CUDA
    assert _call(lib, stride=1032) == pa.PA_ERR_CUDA
    assert _call(lib, bytes=_size(lib)) == pa.PA_ERR_CUDA
    assert _call(lib, hq=256) == pa.PA_ERR_CUDA
    assert _call(lib, cache=dict(kv_tile=1)) == pa.PA_ERR_CUDA
    assert _call(lib, seqs=8192, t=8192, mq=1) == pa.PA_ERR_CUDA


def test_binding_refuses_host_tensors():
    c = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises((ValueError, TypeError, RuntimeError)):
        pa.paged_attention_scored(torch.zeros(1, 8, 128, dtype=torch.bfloat16), c, c, torch.zeros(1, 4, dtype=torch.int32),
                                  i[:1], i, 0.1, 1, 16, out=torch.zeros(1, 8, 128, dtype=torch.bfloat16),
                                  lse=torch.zeros(1, 8), workspace=torch.zeros(256, dtype=torch.uint8))
