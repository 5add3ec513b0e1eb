"""The C-ABI checks of the page calls without a GPU: bad arguments are refused
on the host before any CUDA call, sound ones get as far as CUDA."""
import ctypes

import pytest
import torch

from paged_kv_cache_178_gb300 import build as pa_build
from paged_kv_cache_178_gb300 import pagedattn as pa

INVALID, UNSUPPORTED, OK, WORKSPACE = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_OK, pa.PA_ERR_WORKSPACE

# Aligned addresses 64 MB apart, never dereferenced.
NAMES = ("k", "v", "kk", "vv", "src", "dst", "par", "chi", "len", "ctx", "keep", "bt", "tout", "sin", "sout", "free", "cin",
         "cout", "sl", "cnt", "ws")
AT = {n: (i + 1) << 26 for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real ones")


def _reaches_cuda(rc):
    """A sound call: without a GPU it fails in CUDA; with one it is not issued."""
    return rc == pa.PA_ERR_CUDA


def _kv(**kw):
    c = dict(k=AT["k"], v=AT["v"], num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128, kv_tile=0,
             block_stride=16 * 256, token_stride=256, head_stride=128)
    c.update(kw)
    return pa.PaKvCache(**c)


def _q4(**kw):
    c = dict(k=AT["k"], v=AT["v"], num_blocks=64, block_size=16, num_kv_heads=2, head_dim=128, reserved=0,
             block_stride=2 * 1152, head_stride=1152, k_scale=1.0, v_scale=1.0)
    c.update(kw)
    return pa.PaQuantCache(**c)


def _copy(fn, caches, src=AT["src"], dst=AT["dst"], n=8, count=None):
    kind = type(caches[0])
    return fn((kind * len(caches))(*caches), len(caches) if count is None else count, src, dst, n, None)


def test_copy_refusals(lib):
    for fn, make in ((lib.pa_copy_pages, _kv), (lib.pa_copy_pages_quant, _q4)):
        for kw in (dict(src=0), dict(dst=0), dict(src=AT["src"] + 2), dict(n=-1), dict(n=2**31), dict(count=-1),
                   dict(src=AT["k"]), dict(dst=AT["v"] + 64)):
            assert _copy(fn, [make()], **kw) == INVALID, kw
        assert fn(None, 1, AT["src"], AT["dst"], 8, None) == INVALID
        for other in (dict(num_blocks=63), dict(num_kv_heads=1), dict(head_dim=256, head_stride=9 * 256, token_stride=512),
                      dict(block_stride=16 * 512)):
            c = make()
            for name, x in other.items():
                if hasattr(c, name):
                    setattr(c, name, x)
            assert _copy(fn, [make(), c]) == INVALID, other
        assert _copy(fn, [make()] * 128, n=0) == OK
        assert fn((type(make()) * 129)(*[make()] * 129), 129, AT["src"], AT["dst"], 8, None) == UNSUPPORTED
        assert _copy(fn, [make()], n=0, src=0, dst=0) == OK
        assert fn(None, 0, 0, 0, 8, None) == OK
        assert _copy(fn, [make(block_size=32)]) == UNSUPPORTED
        assert _copy(fn, [make(k=0)]) == INVALID
        assert _copy(fn, [make(), make(v=AT["vv"] + 8)]) == INVALID


@needs_no_gpu
def test_copy_sound_calls(lib):
    second = dict(k=AT["kk"], v=AT["vv"])
    assert _reaches_cuda(_copy(lib.pa_copy_pages, [_kv(), _kv(**second)]))
    assert _reaches_cuda(_copy(lib.pa_copy_pages, [_kv(token_stride=128, head_stride=2048)]))
    assert _reaches_cuda(_copy(lib.pa_copy_pages_quant, [_q4(), _q4(k_scale=2.0, **second)]))


def _fork(lib, **kw):
    a = dict(AT, n=3, b=8, cols=448, blocks=2048, nfree=1000)
    a.update(kw)
    return lib.pa_fork_requests(a["par"], a["chi"], a["len"], a["n"], a["ctx"], a["b"], a["bt"], a["cols"], a["sin"], a["sout"],
                                a["blocks"], a["free"], a["nfree"], a["cin"], a["cout"], a["sl"], a["src"], a["dst"], None)


def _release(lib, **kw):
    a = dict(AT, b=8, cols=448, blocks=2048, nfree=1000)
    a.update(kw)
    return lib.pa_release_pages(a["ctx"], a["keep"], a["b"], a["bt"], a["cols"], a["sin"], a["sout"], a["blocks"], a["free"],
                                a["nfree"], a["cin"], a["cout"], a["sl"], None)


def _compact(lib, **kw):
    a = dict(AT, b=8, cols=448, blocks=2048, nfree=2048, moves=100, bytes=256)
    a.update(kw)
    return lib.pa_compact_pages(a["ctx"], a["b"], a["bt"], a["tout"], a["cols"], a["sin"], a["sout"], a["blocks"], a["free"],
                                a["nfree"], a["cin"], a["cout"], a["src"], a["dst"], a["moves"], a["cnt"], a["ws"], a["bytes"],
                                None)


def test_page_call_refusals(lib):
    for call in (_fork, _release, _compact):
        for kw in (dict(b=-1), dict(cols=0), dict(blocks=0), dict(blocks=2**31 + 1), dict(nfree=-1), dict(ctx=0), dict(bt=0),
                   dict(sin=0), dict(sout=0), dict(free=0), dict(cin=0), dict(cout=0), dict(ctx=AT["ctx"] + 1),
                   dict(bt=AT["bt"] + 2), dict(sout=AT["sin"] + 4), dict(cout=AT["sin"]), dict(sout=AT["ctx"]),
                   dict(free=AT["sout"])):
            assert call(lib, **kw) == INVALID, (call, kw)
        for kw in (dict(b=8193), dict(cols=(2**31 - 1) // 16 + 1), dict(b=8192, cols=262144 + 1)):
            assert call(lib, **kw) == UNSUPPORTED, (call, kw)
        if call is not _fork:  # (a fork only reads the free pages)
            assert call(lib, free=AT["cin"], nfree=4096) == INVALID
    for kw in (dict(n=-1), dict(par=0), dict(chi=0), dict(src=0), dict(dst=0), dict(len=AT["len"] + 1), dict(sl=0),
               dict(sl=AT["ctx"] + 4), dict(src=AT["dst"]), dict(dst=AT["par"]), dict(bt=AT["free"]), dict(b=0),
               dict(sl=AT["len"])):
        assert _fork(lib, **kw) == INVALID, kw
    assert _fork(lib, n=8193) == UNSUPPORTED and _fork(lib, b=0, n=0) == OK
    for kw in (dict(keep=0), dict(sl=0), dict(sl=AT["keep"]), dict(free=AT["bt"] + 64), dict(cout=AT["sl"])):
        assert _release(lib, **kw) == INVALID, kw
    assert _release(lib, b=0, ctx=0) == OK
    for kw in (dict(moves=-1), dict(nfree=2047), dict(src=0), dict(dst=0), dict(cnt=0), dict(tout=0), dict(tout=AT["bt"] + 4),
               dict(src=AT["dst"]), dict(cnt=AT["cout"]), dict(ws=AT["ws"] + 128), dict(ws=AT["free"]), dict(tout=AT["ctx"])):
        assert _compact(lib, **kw) == INVALID, kw
    assert _compact(lib, ws=0) == WORKSPACE and _compact(lib, bytes=255) == WORKSPACE
    assert _compact(lib, blocks=2**20 + 1, nfree=2**20 + 1) == UNSUPPORTED
    size = lib.pa_compact_pages_workspace_size
    assert [size(n) for n in (0, -1, 2**20 + 1, 1, 2048, 2049, 2**20)] == [0, 0, 0, 256, 256, 512, 131072]


@needs_no_gpu
def test_page_call_sound_calls(lib):
    in_place = dict(sl=AT["ctx"], sout=AT["sin"], cout=AT["cin"], tout=AT["bt"])
    for call in (_fork, _release, _compact):
        assert _reaches_cuda(call(lib)) and _reaches_cuda(call(lib, **in_place)), call
    assert _reaches_cuda(_fork(lib, len=0)) and _reaches_cuda(_fork(lib, n=0, par=0, chi=0, src=0, dst=0))
    assert _reaches_cuda(_compact(lib, b=0, ctx=0, bt=0, tout=0)) and _reaches_cuda(_compact(lib, moves=0, src=0, dst=0))
    assert _reaches_cuda(_release(lib, nfree=0, free=0))


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.copy_pages([], t, t)
    with pytest.raises(ValueError):
        pa.release_pages(t, t, t.view(2, 2), t, t, t, t[:1], t[:1], t)
