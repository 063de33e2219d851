"""GPU parity of reading less of a long cache: the operators together as a program uses them, and what they share at the edges."""
import ctypes

import numpy as np
import pytest
import torch

import attn_reference as R
import long_reference as G
from bit_quantized_decode_amd import binding as B
from helpers import device
from test_gpu_attn_shared import Shared
from test_gpu_kv_evict import Weighed

pytestmark = pytest.mark.gpu

WAIT = 2_000_000      # clock ticks, about a millisecond: what follows on that stream is queued behind it


def to(dev, a, dtype=torch.int32):
    return torch.as_tensor(np.array(a, order="C"), dtype=dtype, device=dev)


def rows(n, heads, d, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, d, generator=g).to(torch.bfloat16)


# ---- as they are used together -------------------------------------------------------------------

@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_generation_over_selected_pages(fmt):
    """Each step appends a token, forms the bounds of pages that it fills, selects and attends; the step is one graph."""
    dev, page, hk, hq, d, budget = device(), 16, 2, 6, 64, 5
    lens = np.array([150, 31, 0, 16 * 9 - 1])
    b, width, steps = len(lens), 12, 20
    pages = b * width
    table = np.random.default_rng(1).permutation(pages).reshape(b, width)
    first = np.concatenate([table[i, np.arange(n) // page] * page + np.arange(n) % page for i, n in enumerate(lens)])
    pool = G.Pool(dev, fmt, pages, page, hk, d, seed=2, slots=first, around=1.0)
    full = [table[i, j] for i, n in enumerate(lens) for j in range(n // page)]
    bounds = B.kv_bounds(pool.cache, to(dev, full))
    q, new = (torch.zeros(b, h, d, dtype=torch.bfloat16, device=dev) for h in (hq, 2 * hk))
    slots, filled = torch.zeros(b, dtype=torch.int64, device=dev), torch.full((b,), -1, dtype=torch.int32, device=dev)
    seq, pages_in = torch.zeros(b, dtype=torch.int32, device=dev), to(dev, table)

    def step():
        B.kv_append(pool.cache, new[:, :hk], new[:, hk:], slots)
        B.kv_bounds(pool.cache, filled, bounds)
        chosen, tokens = B.kv_select(q, pool.cache, bounds, pages_in, seq, budget)
        return chosen, tokens, B.attn_decode(q, pool.cache, chosen, tokens, lse=True)

    for t in range(steps):
        at = np.array([table[i, n // page] * page + n % page for i, n in enumerate(lens)])
        k, v = rows(b, hk, d, 100 + t), rows(b, hk, d, 200 + t)
        q.copy_(rows(b, hq, d, 300 + t))
        new[:, :hk], new[:, hk:] = k.to(dev), v.to(dev)
        slots.copy_(torch.from_numpy(at))
        filled.copy_(to(dev, [s // page if s % page == page - 1 else -1 for s in at]))
        lens += 1
        seq.copy_(to(dev, lens))
        if t == 0:
            step()                              # (the same token once more)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step()
        graph.replay()
        torch.cuda.synchronize()
        pool.k[at], pool.v[at] = (R.stored(x.float().numpy(), fmt) for x in (k, v))
        # (Pages that are not full have no bounds yet and are a sequence's last.)
        want, tokens = G.selection(q.cpu(), np.nan_to_num(pool.bounds()), table, lens, budget, page, pages)
        assert np.array_equal(got[0].cpu().numpy(), want) and np.array_equal(got[1].cpu().numpy(), tokens), t
        G.check_rows(pool, q.cpu(), [[pool.slots(want[i, h], tokens[i])[0] for h in range(hk)] for i in range(b)], *got[2], what=t)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_generation_with_eviction(fmt):
    """Steps that weigh their pages; when a table is full, eviction compacts it, its pages serve again, and generation goes on."""
    dev, page, hk, hq, d, width, budget = device(), 16, 2, 6, 64, 8, 5
    lens = np.array([16 * 7 + 9, 40, 16 * 6 + 14])
    b = len(lens)
    pages = b * width
    order = np.random.default_rng(3).permutation(pages)
    table = np.full((b, width), -1, np.int64)
    free = list(order)
    for i, n in enumerate(lens):
        for j in range(-(-n // page)):
            table[i, j] = free.pop()
    first = np.concatenate([table[i, np.arange(n) // page] * page + np.arange(n) % page for i, n in enumerate(lens)])
    pool = G.Pool(dev, fmt, pages, page, hk, d, seed=4, slots=first)
    w, decay = torch.zeros(b, hk, width, device=dev), 0.75
    ref, off = np.zeros((b, hk, width)), np.zeros((b, hk, width))
    evictions = 0
    for t in range(60):
        if (lens == width * page).any():
            before = w.cpu().numpy()
            got = B.kv_evict(w, to(dev, table), to(dev, lens), page, budget, sink=1, recent=2)
            want = G.eviction(before, table, lens, page, budget, 1, 2)
            for g, r in zip(got, want):
                assert np.array_equal(g.cpu().numpy(), r), t
            kept = [[list(table[i]).index(p) for p in want[0][i] if p >= 0] for i in range(b)]
            ref, off = ([np.pad(x[i][:, kept[i]], ((0, 0), (0, width - len(kept[i])))) for i in range(b)] for x in (ref, off))
            ref, off = np.array(ref), np.array(off)
            table = np.pad(want[0], ((0, 0), (0, width - budget)), constant_values=-1)
            lens = want[1].copy()
            w.zero_()
            w[:, :, :budget] = got[3]
            free += [p for p in want[2].reshape(-1) if p >= 0]
            evictions += 1
        for i, n in enumerate(lens):
            if n % page == 0:
                table[i, n // page] = free.pop(0)
        at = np.array([table[i, n // page] * page + n % page for i, n in enumerate(lens)])
        pool.write(at, rows(b, hk, d, 100 + t), rows(b, hk, d, 200 + t))
        lens += 1
        q = rows(b, hq, d, 300 + t)
        out, lse, got = B.attn_weigh(q.to(dev), pool.cache, to(dev, table), to(dev, lens), w, decay, lse=True)
        assert got is w
        G.check_rows(pool, q, [pool.slots(table[i], n)[0] for i, n in enumerate(lens)], out, lse, what=t)
        more, by = G.page_weights(pool, q, table, lens, width)
        ref, off = decay * ref + more, decay * off + by + 2 * R.U24 * (decay * ref + more)
        assert (np.abs(w.double().cpu().numpy() - ref) <= off).all(), t
    assert evictions >= 1 and len(free) == pages - sum(-(-n // page) for n in lens)


@pytest.mark.parametrize("at_once", [False, True], ids=["each", "at_once"])
@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_generation_under_a_shared_prefix(fmt, at_once, monkeypatch):
    """Places of the batch that are free at first, join and leave again; each step appends for those that are there."""
    monkeypatch.setattr(Shared, "at_once", at_once)
    x = Shared(fmt, 100, [-1, 3, -1, 0, 20], 6, 2, 64, 16, seed=21, extra=3)
    dev, page = x.pool.dev, 16
    spare = [p for p in range(x.pool.pages) if p not in set(x.prefix_pages) and p not in set(x.table.reshape(-1))]
    seq, lens = x.args[5], x.lens
    for t in range(24):
        if t == 5:
            lens[0] = 0
        if t == 11:
            lens[4] = -1
        live = [i for i, n in enumerate(lens) if n >= 0]
        for i in live:
            if lens[i] % page == 0 and not 0 <= x.table[i, lens[i] // page] < x.pool.pages:
                if not spare:                   # the pages of a sequence that left
                    spare += [p for p in x.table[4] if 0 <= p < x.pool.pages]
                x.table[i, lens[i] // page] = spare.pop()
        at = np.array([x.table[i, lens[i] // page] * page + lens[i] % page for i in live], np.int64)
        x.pool.write(at, rows(len(at), 2, 64, 100 + t), rows(len(at), 2, 64, 200 + t))
        for i in live:
            lens[i] += 1
        seq.copy_(to(dev, lens))
        x.args[4] = to(dev, x.table)
        x.q = rows(5, 6, 64, 300 + t)
        x.args[0] = x.q.to(dev)
        x.check(what=t)


# ---- scores and values that are not finite, or far apart ------------------------------------------------

def kinds(fmt, lens, seed, qspread=1.0):
    """A batch, and the attentions over it: (name, call -> (out, lse), lists of slots)."""
    page = 32
    x = Weighed(fmt, lens, 4, 2, 64, page, seed=seed, qspread=qspread)
    dev, b = x.dev, len(lens)
    width = x.table.shape[1]
    heads = np.repeat(x.table[:, None], 2, axis=1)
    args = lambda: (x.q.to(dev), x.pool.cache)  # noqa: E731
    out = [("heads", lambda **kw: B.attn_decode(*args(), to(dev, heads), to(dev, lens), lse=True, **kw)),
           ("weigh", lambda **kw: B.attn_weigh(*args(), to(dev, x.table), to(dev, lens), None, 0.0, torch.empty(b, 2, width, device=dev),
                                               lse=True, **kw)[:2])]
    # The first sequence's first two pages as a prefix that all have, those of the others gone.
    own = [max(n - 2 * page, 0) for n in lens]
    rest = to(dev, np.concatenate((x.table[:, 2:], np.full((b, 2), -1)), 1))
    shared = lambda prefix, **kw: B.attn_shared(*args(), to(dev, prefix), to(dev, [min(lens[0], 2 * page)]), rest,  # noqa: E731
                                                to(dev, own), lse=True, **kw)
    out.append(("shared", lambda **kw: shared(x.table[0, :2], **kw)))
    out.append(("shared at once", lambda **kw: shared(G.with_room(x.table[0, :2], fmt, b, 4, 2, 64, page), **kw)))
    whole = [x.pool.slots(x.table[i], n)[0] for i, n in enumerate(lens)]
    first = x.pool.slots(x.table[0, :2], lens[0])[0]
    split = [np.concatenate((first, x.pool.slots(x.table[i, 2:], own[i])[0])) for i in range(b)]
    return x, [(name, call, split if name.startswith("shared") else whole) for name, call in out]


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("at", [3, 70])
def test_nan_in_a_cache_row_stays_in_its_head(fmt, at):
    """In a key: the rows that attend to it are NaN, and their lse.  In a value: the rows (of what its rounding unit holds) and not
    lse.  Place 3 is in the prefix, 70 among the first sequence's own tokens."""
    for side in (0, 1):
        x, calls = kinds(fmt, [200, 50], seed=at)
        bad, ok = torch.ones(1, 2, 64), torch.ones(1, 2, 64)
        bad[0, 1, 5] = float("nan")
        slot = np.array([x.table[0, at // 32] * 32 + at % 32])
        x.pool.write(slot, *((a.to(torch.bfloat16) for a in ((bad, ok) if side == 0 else (ok, bad)))))
        for name, call, lists in calls:
            out, lse = call()
            for b in range(2):
                hit = slot[0] in lists[b]
                assert not out[b, :2].isnan().any() and not lse[b, :2].isnan().any(), (name, b)
                assert out[b, 2:].isnan().any(-1).all() == hit, (name, b)
                assert lse[b, 2:].isnan().all() == (hit and side == 0) and (hit or not lse[b].isnan().any()), (name, b)


class Part:
    """Some heads and channels of a pool."""

    def __init__(self, pool, heads, channels=slice(None)):
        self.fmt, self.k, self.v = pool.fmt, pool.k[:, heads], pool.v[:, heads][..., channels]
        self.hk, self.d = self.k.shape[1:]


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("at", [3, 70])
def test_infinite_keys(at, sign):
    """bf16: a score of -inf weighs nothing, one of +inf makes its query head's row and lse NaN."""
    inf = float("inf")
    x, calls = kinds(B.NVFP4_KV_BF16, [200, 50], seed=at + 1)
    x.q[:, :2, 5], x.q[:, 2:, 5] = sign, -sign                 # head 0: +inf, head 1: -inf
    slot = np.array([x.table[0, at // 32] * 32 + at % 32])
    key = rows(1, 2, 64, 5)
    key[..., 5] = sign * inf
    x.pool.write(slot, key, rows(1, 2, 64, 6))
    for name, call, lists in calls:
        out, lse = call()
        for b in range(2):
            hit = slot[0] in lists[b]
            assert out[b, :2].isnan().all() == hit and lse[b, :2].isnan().all() == hit, (name, b)
        rest = [np.setdiff1d(at_b, slot) for at_b in lists]
        G.check_rows(Part(x.pool, slice(1, 2)), x.q[:, 2:], rest, out[:, 2:], lse[:, 2:], what=name)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_queries_that_are_not_finite(fmt, bad):
    """Their own rows alone: NaN where some score is, nothing where all scores are -inf."""
    x, calls = kinds(fmt, [200, 50], seed=14)
    n = x.pool.pages * 32
    k = rows(n, 2, 64, 7)
    k[:, 1, 5] = -4.0
    x.pool.write(np.arange(n), k, rows(n, 2, 64, 8))
    x.q[0, 2, 5] = bad
    for name, call, lists in calls:
        out, lse = call()
        if bad == bad:
            assert (out[0, 2] == 0).all() and lse[0, 2] == -float("inf"), name
        else:
            assert out[0, 2].isnan().all() and lse[0, 2].isnan(), name
        head = [0, 1, 3]
        for h in head:
            G.check_rows(Part(x.pool, slice(h // 2, h // 2 + 1)), x.q[:, h:h + 1], lists, out[:, h:h + 1], lse[:, h:h + 1], what=(name, h))


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("at", [3, 70])
def test_infinite_values(fmt, at):
    """They reach the outputs that hold them (their element, in E4M3 their row, in NVFP4 their block of 16), and lse not."""
    x, calls = kinds(fmt, [200, 50], seed=15)
    slot = np.array([x.table[0, at // 32] * 32 + at % 32])
    value = rows(1, 2, 64, 9)
    value[0, 1, 5] = float("inf")
    x.pool.write(slot, rows(1, 2, 64, 10), value)
    reach = {0: slice(5, 6), 1: slice(0, 64), 2: slice(0, 16)}[fmt]
    for name, call, lists in calls:
        out, lse = call()
        assert lse.isfinite().all()
        G.check_rows(Part(x.pool, slice(0, 1)), x.q[:, :2], lists, out[:, :2], lse[:, :2], what=name)
        for b in range(2):
            assert out[b, 2:, reach].isfinite().logical_not().all() == (slot[0] in lists[b]), (name, b)
            if fmt != B.NVFP4_KV_E4M3:
                assert out[b, 2:, 16:].isfinite().all()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_garbage_behind_the_last_token_is_not_read(fmt):
    """The places of attended pages that no sequence has reached hold NaN codes and scales (Pool leaves them so)."""
    for lens in ([100, 45], [45, 100], [64, 1]):
        x, calls = kinds(fmt, lens, seed=8)
        for name, call, lists in calls:
            out, lse = call()
            G.check_rows(x.pool, x.q, lists, out, lse, what=name)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_sharp_and_flat_scores(fmt):
    x, calls = kinds(fmt, [900, 64, 63], seed=9, qspread=12.0)
    for scale in (0.5, 1e-6):
        for name, call, lists in calls:
            G.check_rows(x.pool, x.q, lists, *call(scale=scale), scale, (name, scale))


@pytest.mark.parametrize("shift", [24, 32, 90])
def test_scores_far_beyond_the_exponentials_range(shift):
    """Scores of +-2^shift times small integers: all weight on the largest, equal ones share it, in the prefix or not."""
    x, calls = kinds(B.NVFP4_KV_E4M3, [300, 200], seed=10)
    n = x.pool.pages * 32
    k = torch.zeros(n, 2, 64)
    k[:, :, 0] = torch.tensor([2.0, 3.0, 4.0, 6.0])[torch.arange(n) % 4, None]
    v = rows(n, 2, 64, 11)
    x.pool.write(np.arange(n), k.to(torch.bfloat16), v)
    x.q.zero_()
    x.q[:, ::2, 0], x.q[:, 1::2, 0] = 1.0, -1.0
    for name, call, lists in calls:
        out, lse = (t.double().cpu().numpy() for t in call(scale=2.0 ** shift))
        for b in range(2):
            for h in range(4):
                s = float(x.q[b, h, 0]) * x.pool.k[lists[b], h // 2, 0]
                best = x.pool.v[lists[b], h // 2][s == s.max()]
                bound = 2.0 ** -8 * np.abs(best.mean(0)) + (len(best) + 8) * 2.0 ** -24 * np.abs(best).mean(0) + 1e-30
                assert (np.abs(out[b, h] - best.mean(0)) <= bound).all(), (name, b, h)
                assert abs(lse[b, h] - s.max() * 2.0 ** shift) <= 2.0 ** -20 * abs(s.max() * 2.0 ** shift)


@pytest.mark.parametrize("shift", [20, 24, 32, 90])
def test_weights_of_far_scores(shift):
    """Scores of +-2^shift times small integers: pages without a largest term weigh nothing, the others no more than their sixteens."""
    dev, page, n = device(), 32, 300
    x = Weighed(B.NVFP4_KV_E4M3, [n], 4, 2, 64, page, seed=12)
    k = torch.zeros(n, 2, 64)
    best = np.arange(n) // page % 3 == 1                   # pages 1, 4 and 7 hold the largest scores
    k[:, :, 0] = torch.from_numpy(np.where(best & (np.arange(n) % 5 == 0), 6.0, 4.0))[:, None]
    x.pool.write(x.pool.slots(x.table[0], n)[0], k.to(torch.bfloat16), rows(n, 2, 64, 13))
    x.q.zero_()
    x.q[:, :, 0] = 1.0
    w = torch.full((1, 2, x.table.shape[1]), 0.25, device=dev)
    out, lse, w = B.attn_weigh(*x.args(), w, 1.0, scale=2.0 ** shift, lse=True)
    w = w.cpu().numpy() - 0.25
    assert np.isfinite(w).all() and (w[:, :, 0::3] == 0).all() and (w[:, :, 2::3] == 0).all()
    assert (w[:, :, 1::3] >= 0).all() and (w <= 2 * page // 16).all()
    if shift == 20:                                        # half a step of a score is 2^-2: a factor of 2 at most for each rounding
        assert (w[:, :, 1::3] > 0).all()


# ---- the largest -------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_offsets_past_32_bits(fmt):
    """Pages at both ends of a pool of more than 2^32 bytes: prefix, own tokens, bounds, tables of each head, weights."""
    dev, page, hk, d = device(), 64, 8, 128
    group = {0: 8192, 1: 4128, 2: 2304}[fmt]
    pages = (5 << 30) // (group * hk * page // 16)
    cache = B.KvCache(pages, page, hk, d, fmt, device=dev)
    assert cache.pool.numel() > 1 << 32
    ids = np.array([pages - 1, 0, pages // 2, pages - 2])
    n = 4 * page - 5
    j = np.arange(n)
    slots = ids[j // page] * page + j % page
    k, v = rows(n, hk, d, 1), rows(n, hk, d, 2)
    B.kv_append(cache, k.to(dev), v.to(dev), torch.from_numpy(slots).to(dev))

    class Small:                     # the written slots alone, in their order
        pass

    pool = Small()
    pool.fmt, pool.hk, pool.d = fmt, hk, d
    pool.k, pool.v = R.stored(k.float().numpy(), fmt), R.stored(v.float().numpy(), fmt)
    q = rows(1, 2 * hk, d, 3)
    args = (q.to(dev), cache)
    for front in (ids[:2], G.with_room(ids[:2], fmt, 2, 2 * hk, hk, d, page)):
        out, lse = B.attn_shared(q.expand(2, -1, -1).contiguous().to(dev), cache, to(dev, front), to(dev, [2 * page]),
                                 to(dev, np.stack((ids[2:], ids[2:]))), to(dev, [n - 2 * page] * 2), lse=True)
        G.check_rows(pool, q.expand(2, -1, -1), [j, j], out, lse, what="shared")
    out, lse = B.attn_decode(*args, to(dev, np.broadcast_to(ids, (1, hk, 4))), to(dev, [n]), lse=True)
    G.check_rows(pool, q, [j], out, lse, what="heads")
    out, lse, w = B.attn_weigh(*args, to(dev, ids[None]), to(dev, [n]), None, 0.0, torch.empty(1, hk, 4, device=dev), lse=True)
    G.check_rows(pool, q, [j], out, lse, what="weigh")
    assert np.allclose(w.sum(-1).cpu().numpy(), 2.0, atol=1e-4)
    bounds = B.kv_bounds(cache, to(dev, ids[:3]))
    for i, p in enumerate(ids[:3]):
        got, mine = bounds[int(p)].double().cpu().numpy(), pool.k[i * page:(i + 1) * page]
        assert np.array_equal(got[:, 0], mine.min(0)) and np.array_equal(got[:, 1], mine.max(0))
    assert B.kv_select(*args, bounds, to(dev, ids[None]), to(dev, [n]), 4)[0].cpu().tolist() == [[ids.tolist()] * hk]


def test_bounds_offsets_past_32_bits():
    """Bounds of more than 2^32 bytes: the last pages' are written and read where they lie."""
    dev, page, hk, d = device(), 16, 32, 256
    pages = (1 << 32) // (hk * 2 * d * 2) + 100
    cache = B.KvCache(pages, page, hk, d, B.NVFP4_KV_NVFP4, device=dev)
    ids = np.array([pages - 1, 5, pages - 2, 0])
    k = rows(4 * page, hk, d, 1)
    slots = (ids[:, None] * page + np.arange(page)).reshape(-1)
    B.kv_append(cache, k.to(dev), k.to(dev), torch.from_numpy(slots).to(dev))
    bounds = B.kv_bounds(cache, to(dev, ids))
    assert bounds.numel() * 2 > 1 << 32
    stored = R.stored(k.float().numpy(), B.NVFP4_KV_NVFP4).reshape(4, page, hk, d)
    want = np.stack((stored.min(1), stored.max(1)), 2)
    assert np.array_equal(bounds[torch.from_numpy(ids).to(dev)].double().cpu().numpy(), want)
    q = rows(1, hk, d, 2)
    got, _ = B.kv_select(q.to(dev), cache, bounds, to(dev, ids[None]), to(dev, [4 * page]), 2)
    # (`want` by place: the same selection over a table of places.)
    place, _ = G.selection(q, want, np.arange(4)[None], [4 * page], 2, page, 4)
    assert np.array_equal(got.cpu().numpy(), ids[place])


def test_more_workgroups_than_one_row_of_a_grid():
    """Bounds of 40,000 listed pages of 8 heads, weights of 1.2 million pages, joins of 400,000 rows of one token each."""
    dev, page, hk, d = device(), 16, 8, 16
    pool = G.Pool(dev, B.NVFP4_KV_E4M3, 50, page, hk, d, seed=1)
    bounds = torch.full((50, hk, 2, d), 7.0, dtype=torch.bfloat16, device=dev)
    listed = np.full(40_000, -1)
    listed[-50:] = np.arange(50)
    B.kv_bounds(pool.cache, to(dev, listed), bounds)
    assert np.array_equal(bounds.double().cpu().numpy(), pool.bounds())

    b, width = 150, 1000
    lens = np.zeros(b, np.int64)
    lens[[0, 77, 149]] = [3, width * page, 20]
    table = np.random.default_rng(2).integers(0, 50, size=(b, width))
    q = G.queries(b, hk, d)
    w = torch.ones(b, hk, width, device=dev)
    B.attn_weigh(q.to(dev), pool.cache, to(dev, table), to(dev, lens), w, 0.5)
    want, off = G.page_weights(pool, q, table, lens, width)
    assert (np.abs(w.double().cpu().numpy() - 0.5 - want) <= off + 2 * R.U24 * (0.5 + want)).all()

    b = 50_000                      # one page each, of one token; a prefix of one page
    lens = np.ones(b, np.int64)
    lens[1::7] = -1
    table = np.random.default_rng(3).integers(0, 50, size=(b, 1))
    q = G.queries(b, hk, d)
    out, lse = B.attn_shared(q.to(dev), pool.cache, to(dev, [4]), to(dev, [5]), to(dev, table), to(dev, lens), lse=True)
    some = np.concatenate((np.arange(20), np.random.default_rng(4).integers(0, b, 100), np.arange(b - 20, b)))
    first = pool.slots([4], 5)[0]
    lists = [np.concatenate((first, pool.slots(table[i], 1)[0])) if lens[i] >= 0 else first[:0] for i in some]
    G.check_rows(pool, q[some], lists, out[torch.from_numpy(some).to(dev)], lse[torch.from_numpy(some).to(dev)])
    gone = torch.from_numpy(lens < 0).to(dev)
    assert (out[gone] == 0).all() and (lse[gone] == -np.inf).all() and torch.isfinite(out).all()


def test_largest_batch():
    """65,536 places, of which few hold a sequence."""
    dev, page, d, b = device(), 16, 16, 65536
    pool = G.Pool(dev, B.NVFP4_KV_BF16, 60, page, 1, d, seed=5)
    lens = np.full(b, -1)
    live = [0, 1, 40_000, b - 1]
    lens[live] = [40, 0, 17, 48]
    table = np.full((b, 3), -1)
    table[live] = np.arange(12).reshape(4, 3)
    q = G.queries(b, 2, d, seed=6)
    at = torch.tensor(live, device=dev)
    out, lse = B.attn_shared(q.to(dev), pool.cache, to(dev, [50, 51]), to(dev, [30]), to(dev, table), to(dev, lens), lse=True)
    first = pool.slots([50, 51], 30)[0]
    G.check_rows(pool, q[live], [np.concatenate((first, pool.slots(table[i], lens[i])[0])) for i in live], out[at], lse[at])
    lens = np.maximum(lens, 0)
    bounds = B.kv_bounds(pool.cache, to(dev, np.arange(60)))
    chosen, tokens = B.kv_select(q.to(dev), pool.cache, bounds, to(dev, table), to(dev, lens), 2)
    want, want_tokens = G.selection(q[live], pool.bounds(), table[live], lens[live], 2, page, 60)
    assert np.array_equal(chosen[at].cpu().numpy(), want) and np.array_equal(tokens[at].cpu().numpy(), want_tokens)
    assert tokens.sum().item() == want_tokens.sum() and (chosen == -1).sum().item() == chosen.numel() - (want >= 0).sum()
    out, lse = B.attn_decode(q.to(dev), pool.cache, chosen, tokens, lse=True)
    G.check_rows(pool, q[live], [[pool.slots(want[i, 0], want_tokens[i])[0]] for i in range(4)], out[at], lse[at])
    w = torch.ones(b, 1, 3, device=dev)
    B.attn_weigh(q.to(dev), pool.cache, to(dev, table), to(dev, lens), w, 1.0)
    assert abs(w.sum().item() - 3 * b - 6) < 1e-1 and torch.equal(w[1], torch.ones(1, 3, device=dev))
    got = B.kv_evict(w, to(dev, table), to(dev, lens), page, 2, 0, 1)
    ref = G.eviction(w[at].cpu().numpy(), table[live], lens[live], page, 2, 0, 1)
    for g, r in zip(got, ref):
        assert np.array_equal(g[at].cpu().numpy(), r)


@pytest.mark.parametrize("hq,hk", [(32768, 1), (1024, 1024), (32768, 1024)])
def test_most_heads(hq, hk):
    x = Weighed(B.NVFP4_KV_NVFP4, [50], hq, hk, 16, 16, seed=hk)
    x.check(what=(hq, hk))
    bounds = B.kv_bounds(x.pool.cache, to(x.dev, x.table[0, :3]))
    chosen, tokens = B.kv_select(x.q.to(x.dev), x.pool.cache, bounds, to(x.dev, x.table), to(x.dev, [50]), 3)
    want, _ = G.selection(x.q, np.nan_to_num(x.pool.bounds()), x.table, [50], 3, 16, x.pool.pages)
    assert np.array_equal(chosen.cpu().numpy(), want)
    G.check_rows(x.pool, x.q, [[x.pool.slots(want[0, h], tokens.item())[0] for h in range(hk)]],
                 *B.attn_decode(x.q.to(x.dev), x.pool.cache, chosen, tokens, lse=True), what="heads")
    for front in (x.table[0, :2], G.with_room(x.table[0, :2], x.pool.fmt, 1, hq, hk, 16, 16)):
        out, lse = B.attn_shared(x.q.to(x.dev), x.pool.cache, to(x.dev, front), to(x.dev, [32]), to(x.dev, x.table[:, 2:]),
                                 to(x.dev, [18]), lse=True)
        G.check_rows(x.pool, x.q, [x.pool.slots(x.table[0], 50)[0]], out, lse, what="shared")


# ---- streams, graphs, workspaces ----------------------------------------------------------------------

def chain_of(seed=31):
    """(step, inputs): all operators over one cache, from inputs alone; its results."""
    dev = device()
    x = Weighed(B.NVFP4_KV_NVFP4, [3000, 37, 700], 10, 2, 128, 64, seed=seed)
    bounds = torch.zeros(x.pool.pages, 2, 2, 128, dtype=torch.bfloat16, device=dev)
    listed = list(x.table.reshape(-1)) + [p for p in range(x.pool.pages) if p not in x.table]
    inputs = [x.pool.cache.pool, x.q.to(dev), to(dev, x.table), to(dev, x.lens), torch.from_numpy(x.w).to(dev), bounds,
              to(dev, [65]), to(dev, G.with_room(x.table[0, :2], x.pool.fmt, 3, 10, 2, 128, 64)), to(dev, listed), torch.empty(3, 2, x.table.shape[1], device=dev)]

    def chain(stream, pool, q, table, seq, w, bounds, one, front, ids, w2):
        cache = B.KvCache(x.pool.pages, 64, 2, 128, x.pool.fmt, device=dev, pool=pool)
        kw = dict(stream=stream)
        B.kv_bounds(cache, ids, bounds, **kw)
        chosen, tokens = B.kv_select(q, cache, bounds, table, seq, 7, **kw)
        first = B.attn_decode(q, cache, chosen, tokens, lse=True, **kw)
        o, lse, w2 = B.attn_weigh(q, cache, table, seq, w, 0.5, w2, lse=True, **kw)
        shared = B.attn_shared(q, cache, front, one, table, seq, lse=True, **kw)
        by_each = B.attn_shared(q, cache, ids[:2], one, table, seq, lse=True, **kw)
        return (bounds, chosen, tokens, *first, o, lse, w2, *shared, *by_each, *B.kv_evict(w2, table, seq, 64, 9, 1, 2, **kw))

    return chain, inputs


def same(got, want):
    """To the last bit, NaN too (bounds of pages with places that were not written)."""
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_chains_on_overlapping_streams():
    """Three streams, five rounds of all operators each, nothing waited for in between."""
    chain, inputs = chain_of()
    want = [t.clone() for t in chain(None, *(t.clone() for t in inputs))]
    streams = [torch.cuda.Stream() for _ in range(3)]
    mine = [[t.clone() for t in inputs] for _ in streams]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for _ in range(5):
        for s, m, g in zip(streams, mine, got):
            g.append(chain(s, *m))
    torch.cuda.synchronize()
    for g in got:
        for r in g:
            assert same(r, want)


def test_inputs_let_go_while_a_chain_is_queued():
    """Told another stream than the current one; every input is dropped, and its memory asked for again, before it runs."""
    chain, inputs = chain_of()
    want = [t.clone() for t in chain(None, *(t.clone() for t in inputs))]
    s, copies = torch.cuda.Stream(), [t.clone() for t in inputs]
    sizes = [t.numel() * t.element_size() for t in copies]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20 * WAIT)
    got = chain(s, *copies)
    del copies
    taken = [torch.full((n,), 0, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    del taken
    assert same(got, want)


def test_two_graphs_of_the_chain():
    """Captured twice, replayed by turns and on two streams at once, with eager calls between: the same bits."""
    chain, inputs = chain_of()
    want = [t.clone() for t in chain(None, *(t.clone() for t in inputs))]
    graphs, outs, held = [], [], []
    for _ in range(2):
        mine = [t.clone() for t in inputs]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(chain(None, *mine))
        graphs.append(graph)
        held.append(mine)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for step in range(4):
        for out in outs:
            for t in out:
                t.fill_(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
        eager = chain(None, *(t.clone() for t in inputs))
        torch.cuda.synchronize()
        for r in (*outs, eager):
            assert same(r, want), step


def test_prepared_under_capture():
    """Calls prepared inside a capture and called before that graph ever ran, whatever their workspaces hold."""
    x = Weighed(B.NVFP4_KV_BF16, [40 * 64, 0, 700], 10, 2, 128, 64, seed=33)
    dev = x.dev
    q, cache, table, seq = x.args()
    bounds = B.kv_bounds(cache, to(dev, x.table.reshape(-1)))
    many = to(dev, np.tile(x.table[:1, :40], (1, 8)))
    w, w2 = torch.from_numpy(x.w).to(dev), torch.empty(3, 2, x.table.shape[1], device=dev)
    front = to(dev, G.with_room(x.table[0, :9], x.pool.fmt, 3, 10, 2, 128, 64))
    make = [lambda: B.attn_shared_prepared(q, cache, table[0, :9], to_one, table, seq, lse=True),
            lambda: B.attn_shared_prepared(q, cache, front, to_one, table, seq, lse=True),
            lambda: B.kv_select_prepared(q[:1], cache, bounds, many, long, 9),
            lambda: B.attn_weigh_prepared(q, cache, table, seq, w, 0.5, w2, lse=True)]
    to_one, long = to(dev, [500]), to(dev, [320 * 64 - 3])
    for m in make:
        want = [t.clone() for t in m()()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call = m()
            out = call()
        torch.cuda.synchronize()
        ws = next(t for t in reversed(call.keep) if isinstance(t, torch.Tensor) and t.dtype == torch.uint8)
        for step, run in enumerate((call, call, graph.replay, call, graph.replay)):
            for t in out:
                t.fill_(7)
            if step < 3:
                ws[:1024] = 255
            run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), step
        assert not ws[:1024].any()


def test_strided_rows():
    """Queries inside QKV rows and outputs inside wider rows, whose other columns stay as they were."""
    x = Weighed(B.NVFP4_KV_E4M3, [500, 40, 0], 6, 2, 64, 32, seed=34)
    dev, (q, cache, table, seq) = x.dev, x.args()
    wide = torch.full((3, 10, 64), 7.0, dtype=torch.bfloat16, device=dev)
    wide[:, 2:8] = q
    inside = wide[:, 2:8]
    bounds = B.kv_bounds(cache, to(dev, x.table.reshape(-1)))
    bounds[~bounds.isfinite()] = 0.0                     # (of places that were not written)
    chosen, tokens = B.kv_select(q, cache, bounds, table, seq, 4)
    assert all(torch.equal(a, b) for a, b in zip(B.kv_select(inside, cache, bounds, table, seq, 4), (chosen, tokens)))
    w = torch.from_numpy(x.w).to(dev)
    calls = [lambda q, **kw: B.attn_decode(q, cache, chosen, tokens, lse=True, **kw),
             lambda q, **kw: B.attn_weigh(q, cache, table, seq, w, 0.5, torch.empty_like(w), lse=True, **kw)]
    for call in calls:
        want = [t.clone() for t in call(q)]
        out = torch.full((3, 9, 64), 5.0, dtype=torch.bfloat16, device=dev)
        got = call(inside, out=out[:, 1:7])
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(out[:, 1:7], want[0])
        assert (out[:, 0] == 5).all() and (out[:, 7:] == 5).all()


def test_eviction_without_freed_pages_and_weights():
    """The C call with neither: table and lengths alone; and with each of them alone."""
    dev, width, budget = device(), 40, 7
    rng = np.random.default_rng(35)
    weights = rng.exponential(size=(3, 2, width)).astype(np.float32)
    table, lens = rng.permutation(3 * width).reshape(3, width), [width * 16, 100, 0]
    want = G.eviction(weights, table, lens, 16, budget, 1, 2)
    w, t, n = torch.from_numpy(weights).to(dev), to(dev, table), to(dev, lens)
    for with_freed in (False, True):
        for with_weights in (False, True):
            got = [torch.full(s, 7, dtype=d, device=dev) for s, d in (((3, budget), torch.int32), ((3,), torch.int32),
                                                                      ((3, width), torch.int32), ((3, 2, budget), torch.float32))]
            a = B.KvEvictArgs(batch=3, kv_heads=2, page_size=16, weights=w.data_ptr(), page_table=t.data_ptr(), table_width=width,
                              seq_lens=n.data_ptr(), budget=budget, sink=1, recent=2, table_out=got[0].data_ptr(),
                              lens_out=got[1].data_ptr(), freed=got[2].data_ptr() if with_freed else None,
                              weights_out=got[3].data_ptr() if with_weights else None)
            B.check(B.lib().nvfp4_kv_evict(ctypes.byref(a), torch.cuda.current_stream().cuda_stream))
            torch.cuda.synchronize()
            for i, there in enumerate((True, True, with_freed, with_weights)):
                assert np.array_equal(got[i].cpu().numpy(), want[i]) if there else (got[i] == 7).all(), i


def test_a_stream_of_another_device():
    dev = device()

    class Elsewhere:
        device, cuda_stream = torch.device("cuda", torch.cuda.device_count()), 0

    s = Elsewhere()
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device=dev)
    q, i32 = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    bounds, w = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device=dev), torch.zeros(2, 1, 1, device=dev)
    table = i32[:, None].contiguous()
    for call in (lambda: B.attn_shared(q, cache, i32, i32[:1], table, i32, stream=s), lambda: B.kv_bounds(cache, i32, stream=s),
                 lambda: B.kv_select(q, cache, bounds, table, i32, 2, stream=s),
                 lambda: B.attn_weigh(q, cache, table, i32, w, stream=s),
                 lambda: B.kv_evict(w, table, i32, 16, 1, stream=s)):
        with pytest.raises(ValueError, match="stream is on"):
            call()
