"""One workspace for calls of every kind on the attention side, in turn."""
import ctypes

import numpy as np
import pytest
import torch

import long_reference as G
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu


def to(dev, a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device=dev)


def many_pairs(fmt, batch=16, heads=32, d=128, page=16, width=200, seed=1):
    """`batch` ragged sequences of `heads` ungrouped heads over a pool of few pages, each of them used many times: (sequence, kv
    head)s enough for counters past the first kilobyte, tables long enough to be cut over workgroups."""
    dev = device()
    rng = np.random.default_rng(seed)
    pool = G.Pool(dev, fmt, 64, page, heads, d, seed)
    table = to(dev, rng.integers(0, 64, size=(batch, width)))
    lens = rng.integers(1, width * page + 1, size=batch)
    lens[0] = width * page
    bounds = B.kv_bounds(pool.cache, to(dev, np.arange(64)))
    return pool, G.queries(batch, heads, d, seed + 1).to(dev), table, to(dev, lens), bounds


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_attentions_and_selections_share_a_workspace(fmt):
    """Attention leaves the counters of selections as they were, and so both may have one workspace."""
    pool, q, table, lens, bounds = many_pairs(fmt)
    dev, cache, (batch, heads, d) = pool.dev, pool.cache, q.shape
    w = torch.zeros(batch, heads, table.shape[1], device=dev)
    front = to(dev, G.with_room(np.arange(3), fmt, batch, heads, heads, d, 16))
    attentions = [lambda **kw: B.attn_decode(q, cache, table, lens, **kw),
                  lambda **kw: B.attn_weigh(q, cache, table, lens, None, 0.0, w, **kw),
                  lambda **kw: B.attn_shared(q, cache, front[:3], lens[:1] * 0 + 40, table, lens, **kw),
                  lambda **kw: B.attn_shared(q, cache, front, lens[:1] * 0 + 40, table, lens, **kw)]
    want = [t.clone() for t in B.kv_select(q, cache, bounds, table, lens, 9)]
    ws = torch.zeros(96 << 20, dtype=torch.uint8, device=dev)
    for round in range(2):
        for i, attention in enumerate(attentions):
            attention(ws=ws)
            torch.cuda.synchronize()
            assert not ws[:B.NVFP4_SELECT_COUNTER_BYTES].any(), (round, i)
            out = [torch.full_like(t, -7) for t in want]
            B.kv_select(q, cache, bounds, table, lens, 9, *out, ws=ws)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (round, i)
            assert not ws[:B.NVFP4_SELECT_COUNTER_BYTES].any(), (round, i)


@pytest.mark.parametrize("batch", [1, 5])
def test_eviction_leaves_a_workspace_as_others_need_it(batch):
    """Keys of tables beyond 8192 pages lie in the workspace: whatever it held, its front is zero afterwards, or as it was where
    nothing needed keys there; attention and selection may have it next."""
    dev, hk, width, page, budget = device(), 2, 9001, 16, 700
    rng = np.random.default_rng(batch)
    weights = torch.from_numpy(rng.exponential(size=(batch, hk, width)).astype(np.float32)).to(dev)
    table = to(dev, rng.integers(0, 1 << 20, size=(batch, width)))
    pool, q, other, seq, bounds = many_pairs(B.NVFP4_KV_NVFP4)
    w = torch.zeros(16, 32, other.shape[1], device=dev)
    attend = lambda **kw: B.attn_weigh(q, pool.cache, other, seq, None, 0.0, w, lse=True, **kw)  # noqa: E731
    select = lambda **kw: B.kv_select(q, pool.cache, bounds, other, seq, 9, **kw)  # noqa: E731
    want = [t.clone() for t in (*attend(), *select())]
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    for longest in (width * page, 8192 * page, 40, width * page - 3):
        lens = to(dev, [longest] + [rng.integers(0, width * page) for _ in range(batch - 1)])
        ref = B.kv_evict(weights, table, lens, page, budget, 1, 2)
        got = [torch.full_like(t, -7) for t in ref]
        a = B.KvEvictArgs(batch=batch, kv_heads=hk, page_size=page, weights=weights.data_ptr(), page_table=table.data_ptr(),
                          table_width=width, seq_lens=lens.data_ptr(), budget=budget, sink=1, recent=2, table_out=got[0].data_ptr(),
                          lens_out=got[1].data_ptr(), freed=got[2].data_ptr(), weights_out=got[3].data_ptr(),
                          workspace=ws.data_ptr(), workspace_bytes=ws.numel())
        B.check(B.lib().nvfp4_kv_evict(ctypes.byref(a), torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, ref)), longest
        assert not ws[:B.NVFP4_SELECT_COUNTER_BYTES].any(), longest
        assert all(torch.equal(x, y) for x, y in zip((*attend(ws=ws), *select(ws=ws)), want)), longest


def test_selections_prepared_under_capture_clear_all_their_counters():
    """More than 256 and fewer than 1024 (sequence, kv head)s, tables cut over workgroups: counters past the first kilobyte.
    Whatever the workspace holds when a call comes that was prepared inside a capture, and before that graph ever ran."""
    pool, q, table, lens, bounds = many_pairs(B.NVFP4_KV_E4M3, seed=5)
    make = lambda: B.kv_select_prepared(q, pool.cache, bounds, table, lens, 9)  # noqa: E731
    want = [t.clone() for t in make()()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call = make()
        out = call()
    torch.cuda.synchronize()
    ws = next(t for t in reversed(call.keep) if isinstance(t, torch.Tensor) and t.dtype == torch.uint8)
    for step, run in enumerate((call, call, graph.replay, call, graph.replay)):
        for t in out:
            t.fill_(7)
        ws[:B.NVFP4_SELECT_COUNTER_BYTES] = 255
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), step
        assert not ws[:B.NVFP4_SELECT_COUNTER_BYTES].any(), step
