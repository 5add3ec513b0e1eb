"""The step operators as they are used together, on one stream and in one
captured graph: metadata from lengths, norm and rotation, the write into the
4-bit cache, attention over it."""
import numpy as np
import pytest
import torch

from paged_kv_cache_178_gb300 import pagedattn as pa
from tests import step_reference as ref
from tests.helpers import bits, bits_to_f64

pytestmark = pytest.mark.gpu

HQ, HKV, DH, B = 8, 2, 128, 3


def _f64(t):
    return bits_to_f64(bits(t))


class Model:
    """One layer's state and the four calls of a step."""

    def __init__(self, num_blocks=64, max_blocks=12, stream=None):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.stream = stream
        self.cache = pa.new_quant_cache(num_blocks, HKV, DH, 0.5, 1.0)
        self.num_blocks = num_blocks
        self.lens, self.cursor = torch.zeros(B, **i32), torch.zeros(1, **i32)
        self.tables = torch.full((B, max_blocks), -1, **i32)
        self.free = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.table = pa.rope_table(256, DH, device="cuda")
        g = torch.Generator().manual_seed(2)
        self.w = [(1 + 0.2 * torch.randn(DH, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
        self.starts = torch.zeros(B + 1, **i32)

    def calls(self, tokens, new, max_q):
        """The calls of a step of up to `tokens` tokens, max_q per request."""
        self.new = new
        self.qkv = torch.zeros(tokens, (HQ + 2 * HKV) * DH, dtype=torch.bfloat16, device="cuda")
        q, k, v = (x.view(tokens, -1, DH) for x in self.qkv.split([HQ * DH, HKV * DH, HKV * DH], 1))
        self.slots = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        self.pos = torch.zeros(tokens, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(tokens, HQ, DH, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(tokens, HQ, device="cuda")
        cap = self.tables.shape[1] * 16
        ws = pa.new_quant_workspace(B, HQ, HKV, DH, max_q, cap, device="cuda")
        st = dict(stream=self.stream)
        return [pa.prepare_build_step_metadata(self.lens, new, self.tables, self.free, self.num_blocks, self.slots,
                                               self.pos, self.lens, self.starts, self.cursor, self.cursor, **st),
                pa.prepare_qk_norm_rope(q, k, self.pos, self.table, q, k, self.w[0], self.w[1], **st),
                pa.prepare_reshape_and_cache_quant(k, v, self.cache, self.slots, **st),
                pa.prepare_paged_attention_quant(q, self.cache, self.tables, self.lens, self.starts, DH ** -0.5, max_q,
                                                 cap, self.out, self.lse, ws, **st)]


def _reference_step(history, qkv, new, w):
    """Plain 64-bit step over each request's kept K and V; the rotated k and q
    are rounded to BF16 and K, V to 4 bits where the operators round."""
    bf16 = lambda x: torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    table = pa.rope_table(256, DH).numpy()
    outs, at = [], 0
    for b, n in enumerate(new):
        x = qkv[at:at + n]
        at += n
        q, k, v = (y.reshape(n, -1, DH) for y in np.split(x, [HQ * DH, (HQ + HKV) * DH], 1))
        pos = len(history[b][0]) + np.arange(n)
        q = bf16(ref.norm_rope(q, w[0], 0.0, 1e-6, pos, table, False)[0])
        k = bf16(ref.norm_rope(k, w[1], 0.0, 1e-6, pos, table, False)[0])
        k, v = ref.values(*ref.quantise(k, 0.5), 0.5), ref.values(*ref.quantise(v, 1.0), 1.0)
        history[b] = (np.concatenate([history[b][0], k]), np.concatenate([history[b][1], v]))
        kk, vv = (np.repeat(h, HQ // HKV, 1) for h in history[b])
        z = np.einsum("ihd,jhd->hij", q, kk) * DH ** -0.5
        for i in range(n):
            z[:, i, len(kk) - n + i + 1:] = -np.inf
        p = np.exp(z - z.max(-1, keepdims=True))
        outs.append(np.einsum("hij,jhd->ihd", p / p.sum(-1, keepdims=True), vv))
    return np.concatenate(outs)


def _close(got, want):
    # the operators' k differs from the reference's by at most one BF16 step in
    # a few elements, which can move a 4-bit code (a sixth of its block's
    # largest at most); one such key among n moves an output by a small share
    err = np.abs(_f64(got) - want)
    assert np.linalg.norm(err) <= 1e-2 * np.linalg.norm(want), np.linalg.norm(err) / np.linalg.norm(want)


def test_prompt_then_decode_graph_replays():
    s = torch.cuda.Stream()
    pa.init()
    m = Model(stream=s)
    w = [_f64(x) for x in m.w]
    gen = torch.Generator().manual_seed(5)
    empty = np.zeros((0, HKV, DH))
    history = [(empty, empty) for _ in range(B)]
    # prompts of 37, 16 and 1 tokens in one padded call
    lens = [37, 16, 1]
    new = torch.tensor(lens, dtype=torch.int32, device="cuda")
    calls = m.calls(60, new, 37)
    x = torch.randn(60, m.qkv.shape[1], generator=gen).to(torch.bfloat16)
    m.qkv.copy_(x)
    m.out.fill_(7.0)
    torch.cuda.synchronize()
    for c in calls:
        c()
    s.synchronize()
    assert pa.check_errors(s) == (pa.PA_OK, -1)
    _close(m.out[:54], _reference_step(history, _f64(x)[:54], lens, w))
    assert bool((m.out[54:] == 7).all()) and m.lens.tolist() == lens
    # twenty decode steps: one graph, its own lengths and pages advancing
    calls = m.calls(B, torch.ones(B, dtype=torch.int32, device="cuda"), 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for c in calls:
            c()
    for step in range(20):
        x = torch.randn(B, m.qkv.shape[1], generator=gen).to(torch.bfloat16)
        with torch.cuda.stream(s):
            m.qkv.copy_(x)
            g.replay()
        s.synchronize()
        _close(m.out, _reference_step(history, _f64(x), [1] * B, w))
    assert m.lens.tolist() == [n + 20 for n in lens]
    assert int(m.cursor) == sum(-(-(n + 20) // 16) for n in lens)
    assert pa.check_errors(s) == (pa.PA_OK, -1)


def test_step_without_pages_changes_nothing():
    """When the free pages run out the whole chain is an empty step."""
    m = Model(num_blocks=64)
    calls = m.calls(8, torch.full((B,), 2, dtype=torch.int32, device="cuda"), 2)
    for c in calls:
        c()
    assert pa.check_errors() == (pa.PA_OK, -1)
    m.cursor.fill_(64)          # no free page left; the next step needs new ones
    m.lens.fill_(16)
    pool = m.cache.k_pool.clone()
    m.out.fill_(7.0)
    for c in calls:
        c()
    st, idx = pa.check_errors()
    assert (st, idx) == (pa.PA_ERR_WORKSPACE, 3)
    assert torch.equal(pool, m.cache.k_pool) and bool((m.out == 7).all()) and m.lens.tolist() == [16] * 3
