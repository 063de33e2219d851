"""GPU parity: attention of a batch over a prefix that all its sequences share, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import long_reference as G
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu


class Shared:
    at_once = False       # whether the prefix's table has room for a prefix that is read for all sequences at once

    def __init__(self, fmt, prefix, lens, hq, hk, d, page, seed=0, scales=(1.0, 1.0), qspread=1.0, extra=0):
        dev = device()
        rng = np.random.default_rng(seed)
        self.prefix, self.lens = prefix, list(lens)
        b, first = len(lens), -(-prefix // page)
        width = max([1] + [-(-n // page) for n in lens]) + extra
        pages = first + b * width + 2
        order = rng.permutation(pages)
        self.prefix_pages = order[:first].astype(np.int32)
        self.table = np.full((b, width), 2 ** 31 - 1, np.int32)
        at = first
        slots = [self.prefix_pages[np.arange(prefix) // page].astype(np.int64) * page + np.arange(prefix) % page]
        for i, n in enumerate(lens):
            used = max(0, -(-n // page))
            self.table[i, :used] = order[at:at + used]
            at += used
            slots.append(self.table[i, np.arange(max(n, 0)) // page].astype(np.int64) * page + np.arange(max(n, 0)) % page)
        self.pool = G.Pool(dev, fmt, pages, page, hk, d, seed, scales, slots=np.concatenate(slots))
        self.q = G.queries(b, hq, d, seed + 1, qspread)
        if self.at_once:
            self.prefix_pages = G.with_room(self.prefix_pages, fmt, b, hq, hk, d, page)
        self.args = [self.q.to(dev), self.pool.cache, torch.from_numpy(self.prefix_pages).to(dev),
                     torch.tensor([prefix], dtype=torch.int32, device=dev), torch.from_numpy(self.table).to(dev),
                     torch.tensor(self.lens, dtype=torch.int32, device=dev)]

    def lists(self, prefix=None):
        first, _ = self.pool.slots(self.prefix_pages, self.prefix if prefix is None else prefix)
        return [np.concatenate((first, self.pool.slots(self.table[b], n)[0])) if n >= 0 else np.zeros(0, np.int64)
                for b, n in enumerate(self.lens)]

    def check(self, what="", **kw):
        out, lse = B.attn_shared(*self.args, lse=True, **kw)
        G.check_rows(self.pool, self.q, self.lists(), out, lse, kw.get("scale"), what)
        return out, lse


@pytest.fixture(autouse=True, params=[False, True], ids=["each", "at_once"])
def at_once(request, monkeypatch):
    monkeypatch.setattr(Shared, "at_once", request.param)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 31, 33, 64, 100, 128, 129, 1000, 4097])
def test_prefix_lengths(fmt, prefix):
    Shared(fmt, prefix, [5, 1, 70], 10, 2, 128, 64, seed=prefix).check()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("d", [16, 48, 64, 80, 96, 128, 160, 192, 208, 256])
def test_head_sizes(fmt, d):
    """Three, 24 and 44 rows a kv head: one, two and three row tiles."""
    for users in (1, 8, 14):
        Shared(fmt, 300, [(7 * i) % 40 for i in range(users)], 6, 2, d, 32, seed=d + users).check(what=(d, users))


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 7), (8, 4), (5, 1), (16, 1), (17, 1), (40, 1), (66, 2)])
@pytest.mark.parametrize("users", [1, 3, 16, 37])
def test_rows(fmt, hq, hk, users):
    """1 to 1480 rows a kv head, blocks of rows that end inside a tile and inside a sequence's heads."""
    Shared(fmt, 200, [i % 5 for i in range(users)], hq, hk, 64, 16, seed=hq + users).check(what=(hq, hk, users))


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("page", [16, 48, 80, 1024])
def test_page_sizes(fmt, page):
    Shared(fmt, 3 * page + 7, [1, page - 1, page, page + 1, 2 * page + 5], 4, 2, 64, page, seed=page).check(what=page)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("prefix", [0, 77])
def test_free_places_and_sequences_without_tokens(fmt, prefix):
    """A length of 0 attends to the prefix alone, one below 0 to nothing; rows of nothing are zeros and -inf."""
    x = Shared(fmt, prefix, [0, -1, 9, -2 ** 31, 0, 40], 4, 2, 64, 32, seed=3)
    out, lse = x.check()
    for b in (1, 3):
        assert (out[b] == 0).all() and (lse[b] == -np.inf).all()
    assert ((out[0] == 0).all()) == (prefix == 0)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_lengths_beyond_the_tables(fmt):
    """A prefix length past its table, or below 0, is taken to the table's end and to 0; so are own lengths past theirs."""
    x = Shared(fmt, 96, [32, 64], 4, 2, 64, 32, seed=4)
    for n, want in ((10 ** 9, 96), (-5, 0), (97, 96), (40, 40)):
        x.args[3] = torch.tensor([n], dtype=torch.int32, device=x.pool.dev)
        out, lse = B.attn_shared(*x.args, lse=True)
        G.check_rows(x.pool, x.q, x.lists(want), out, lse, what=n)
    # No prefix table at all.
    x.args[2], x.args[3] = x.args[2][:0], torch.tensor([50], dtype=torch.int32, device=x.pool.dev)
    out, lse = B.attn_shared(*x.args, lse=True)
    G.check_rows(x.pool, x.q, x.lists(0), out, lse)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_evicted_pages(fmt):
    """Pages outside the pool, of the prefix and of a sequence, hold nothing: whole tiles, halves of tiles, and all of it."""
    x = Shared(fmt, 16 * 9 + 3, [70, 3], 4, 2, 64, 16, seed=5)
    for gone in ([0], [1, 2], [8, 9], [3, 4, 5, 6], list(range(10))):
        pages = x.prefix_pages.copy()
        pages[gone] = [(-1, 2 ** 31 - 1, x.pool.pages)[i % 3] for i in range(len(gone))]
        y = list(x.args)
        y[2] = torch.from_numpy(pages).to(x.pool.dev)
        out, lse = B.attn_shared(*y, lse=True)
        first, _ = x.pool.slots(pages, x.prefix)
        lists = [np.concatenate((first, x.pool.slots(x.table[b], n)[0])) for b, n in enumerate(x.lens)]
        G.check_rows(x.pool, x.q, lists, out, lse, what=gone)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_the_prefix_may_be_a_sequences_own_too(fmt):
    """Pages listed twice: the prefix read twice by one sequence, its tokens counting twice."""
    x = Shared(fmt, 64, [64, 10], 4, 2, 64, 32, seed=6)
    x.table[0, :2] = x.prefix_pages[:2]
    x.args[4] = torch.from_numpy(x.table).to(x.pool.dev)
    x.check()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_scales_and_softmax_scale(fmt):
    scales = (0.037, 3.1) if fmt == B.NVFP4_KV_NVFP4 else (1.0, 1.0)
    x = Shared(fmt, 500, [40, 1, 0], 8, 2, 128, 32, seed=7, scales=scales, qspread=4.0)
    x.check(scale=0.5)
    x.check(scale=1e-3)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_long_prefix_of_many_rows(fmt):
    """Cuts of the prefix over all workgroups, several units a workgroup and several workgroups a unit."""
    Shared(fmt, 20011, [3, 0, 129], 8, 2, 64, 64, seed=8).check()
    Shared(fmt, 40, [i % 3 for i in range(300)], 12, 3, 64, 16, seed=9).check()
    Shared(fmt, 1500, [i % 3 for i in range(64)], 15, 3, 128, 16, seed=10).check()
    Shared(fmt, 700, [i % 40 for i in range(9)], 160, 4, 64, 32, seed=10).check()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_strided_rows(fmt):
    """Queries inside QKV rows, outputs inside wider rows whose other columns stay as they were."""
    x = Shared(fmt, 130, [20, 3, 50], 4, 2, 64, 32, seed=11)
    dev = x.pool.dev
    wide = torch.full((3, 8, 64), 7.0, dtype=torch.bfloat16, device=dev)
    wide[:, :4] = x.args[0]
    x.args[0] = wide[:, :4]
    out = torch.full((3, 6, 64), 5.0, dtype=torch.bfloat16, device=dev)
    x.check(out=out[:, 1:5])
    assert (out[:, 0] == 5).all() and (out[:, 5] == 5).all()


def test_same_bits_each_time_and_shared_workspace():
    """Repeated calls, with other attention on the same workspace in between, give the same bits; the counters stay zero."""
    x = Shared(B.NVFP4_KV_NVFP4, 3000, [400, 30, 0, 7], 10, 2, 128, 64, seed=12)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=x.pool.dev)
    out, lse = (t.clone() for t in B.attn_shared(*x.args, lse=True, ws=ws))
    for _ in range(5):
        B.attn_decode(x.args[0], x.pool.cache, x.args[4], x.args[5].clamp(min=0), ws=ws)
        o, l = B.attn_shared(*x.args, lse=True, ws=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)
        assert (ws[:B.NVFP4_ATTN_COUNTER_BYTES] == 0).all()


def test_prepared_streams_and_graphs():
    x = Shared(B.NVFP4_KV_E4M3, 700, [40, 3, 0], 8, 2, 64, 32, seed=13)
    dev = x.pool.dev
    out, lse = x.check()
    call = B.attn_shared_prepared(*x.args, lse=True)
    assert all(torch.equal(a, b) for a, b in zip(call(), (out, lse)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = B.attn_shared(*x.args, stream=side)
    side.synchronize()
    assert torch.equal(o2, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = B.attn_shared(*x.args, lse=True)
    for n in (700, 33, 0, 640):             # the prefix grows and shrinks between replays
        x.args[3].fill_(n)
        want = x.lists(n)
        eager = B.attn_shared(*x.args, lse=True)
        og.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, eager[0]) and torch.equal(lg, eager[1])
        G.check_rows(x.pool, x.q, want, og, lg, what=n)
