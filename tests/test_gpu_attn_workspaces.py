"""One workspace for calls of every kind on the attention side, in turn."""
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
