"""GPU parity: attention that weighs the pages it reads, and eviction by those weights, against the definitions."""
import numpy as np
import pytest
import torch

import attn_reference as R
import long_reference as G
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu


def to(dev, a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device=dev)


class Weighed:
    def __init__(self, fmt, lens, hq, hk, d, page, seed=0, scales=(1.0, 1.0), extra=0, qspread=1.0):
        self.dev = device()
        rng = np.random.default_rng(seed)
        self.lens, width = list(lens), max([1] + [-(-n // page) for n in lens]) + extra
        b = len(lens)
        pages = b * width + 1
        self.table = rng.permutation(pages)[:b * width].reshape(b, width)
        slots = np.concatenate([np.zeros(0, np.int64)] + [self.table[i, np.arange(max(n, 0)) // page] * page + np.arange(max(n, 0)) % page
                                                          for i, n in enumerate(lens)])
        self.pool = G.Pool(self.dev, fmt, pages, page, hk, d, seed, scales, slots=slots)
        self.q = G.queries(b, hq, d, seed + 1, qspread)
        self.w = rng.exponential(size=(b, hk, width)).astype(np.float32)

    def args(self):
        return self.q.to(self.dev), self.pool.cache, to(self.dev, self.table), to(self.dev, self.lens)

    def check(self, decay=0.75, window=0, scale=None, what="", **kw):
        w = torch.from_numpy(self.w).to(self.dev)
        out, lse, got = B.attn_weigh(*self.args(), w, decay, torch.full_like(w, -7.0), scale, window, lse=True, **kw)
        assert torch.equal(w.cpu(), torch.from_numpy(self.w))
        lists = [self.pool.slots(self.table[b], n, max(0, n - window) if window else 0)[0] for b, n in enumerate(self.lens)]
        G.check_rows(self.pool, self.q, lists, out, lse, scale, what)
        want, off = G.page_weights(self.pool, self.q, self.table, self.lens, self.w.shape[2], scale, window)
        kept = np.float64(np.float32(decay)) * self.w
        err, bound = np.abs(got.double().cpu().numpy() - kept - want), off + 2 * R.U24 * (kept + want)
        assert (err <= bound).all(), (what, (err / bound).max(), np.unravel_index((err / bound).argmax(), err.shape))
        return out, lse, got


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 100, 129, 1000, 4097])
def test_lengths(fmt, n):
    Weighed(fmt, [n], 10, 2, 128, 64, seed=n, extra=n % 3).check()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("d", [16, 48, 64, 96, 128, 160, 192, 208, 256])
def test_head_sizes(fmt, d):
    Weighed(fmt, [70, 300, 0, 5], 6, 2, d, 32, seed=d).check()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 7), (8, 4), (16, 1), (17, 1), (40, 1), (66, 2)])
def test_head_groups(fmt, hq, hk):
    Weighed(fmt, [200, 0, 33], hq, hk, 64, 16, seed=hq).check()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("page", [16, 48, 80, 128, 1024])
@pytest.mark.parametrize("window", [0, 1, 7, 16, 100, 500, 10 ** 12])
def test_pages_and_windows(fmt, page, window):
    """Pages that the window's start cuts, that lie outside it, and that tiles straddle; 16 and 64 lanes a page."""
    Weighed(fmt, [1, page - 1, page, page + 1, 3 * page + 7, 777], 10, 2, 64, page, seed=page).check(window=window, what=(page, window))


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_long_and_many(fmt):
    """Units cut over wavefronts and workgroups; large and small scores; tensor scales."""
    scales = (0.037, 3.1) if fmt == B.NVFP4_KV_NVFP4 else (1.0, 1.0)
    Weighed(fmt, [70001], 8, 1, 64, 64, seed=1, scales=scales).check()
    Weighed(fmt, [9000, 1, 100, 4000], 8, 2, 64, 64, seed=2, qspread=6.0).check(scale=0.5)
    Weighed(fmt, list(np.random.default_rng(3).integers(0, 300, size=100)), 6, 2, 64, 32, seed=3).check()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_evicted_pages_and_empty_rows(fmt):
    """Pages that are gone add nothing (their weights only decay), nor do rows without a token; decay 0 and 1."""
    x = Weighed(fmt, [100, 64, 0, 40], 4, 2, 64, 16, seed=4)
    x.table[0, [0, 3]], x.table[1, :] = -1, x.pool.pages
    for decay in (1.0, 0.0, 0.5):
        out, lse, w = x.check(decay)
        assert torch.equal(w[1:3].cpu(), torch.from_numpy(x.w[1:3] * np.float32(decay)))
        assert (out[1] == 0).all() and (lse[1] == -np.inf).all()


def test_weights_in_place_and_without_any():
    """By default weights are updated; with decay 0 they are not read (NaN) and may be missing; lse may be too."""
    x = Weighed(B.NVFP4_KV_NVFP4, [100, 40], 4, 2, 64, 16, seed=5)
    w = torch.from_numpy(x.w).to(x.dev)
    out, lse, want = x.check(1.0)
    o, got = B.attn_weigh(*x.args(), w)
    assert got is w and torch.equal(w, want) and torch.equal(o, out)
    _, _, want = x.check(0.0)
    w.fill_(float("nan"))
    assert torch.equal(B.attn_weigh(*x.args(), w, 0.0)[1], want)
    w.fill_(float("nan"))
    assert torch.equal(B.attn_weigh(*x.args(), None, 0.0, w)[1], want)
    # Every query head's share adds up to 1.
    assert np.allclose(want.sum(-1).cpu().numpy(), 2.0, atol=1e-5)


def test_nan_and_infinite_scores():
    """A query head whose lse is NaN makes its kv head's attended pages NaN and no others."""
    x = Weighed(B.NVFP4_KV_BF16, [40, 70], 4, 2, 64, 16, seed=6, extra=1)
    x.q[0, 3, 5] = float("nan")
    w = torch.from_numpy(x.w).to(x.dev)
    _, lse, got = B.attn_weigh(*x.args(), w, 1.0, torch.empty_like(w), lse=True)
    got = got.cpu().numpy()
    assert np.isnan(got[0, 1, :3]).all() and np.array_equal(got[0, 1, 3:], x.w[0, 1, 3:])
    assert not np.isnan(got[0, 0]).any() and not np.isnan(got[1]).any()


def test_same_as_attn_decode():
    """out and lse are attn_decode()'s to the last bit."""
    for fmt in G.FORMATS:
        x = Weighed(fmt, [5000, 3, 0, 700], 10, 2, 128, 64, seed=7)
        o, l, _ = x.check()
        o2, l2 = B.attn_decode(*x.args(), lse=True)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_calls_of_all_kinds():
    """Repeated, prepared, on another stream, captured: the same bits, the counters left zero."""
    x = Weighed(B.NVFP4_KV_E4M3, [3000, 3, 0, 700], 10, 2, 64, 64, seed=8)
    want = x.check(0.5)
    w = torch.from_numpy(x.w).to(x.dev)
    args = (*x.args(), w, 0.5, torch.empty_like(w))
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device=x.dev)
    prepared = B.attn_weigh_prepared(*args, lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for got in (B.attn_weigh(*args, lse=True, ws=ws), prepared(), B.attn_weigh(*args, lse=True, stream=side)):
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (ws[:B.NVFP4_ATTN_COUNTER_BYTES] == 0).all()
    graph = torch.cuda.CUDAGraph()
    acc = w.clone()
    with torch.cuda.graph(graph):
        B.attn_weigh(*args[:4], acc, 0.5, lse=True)
    eager = w.clone()
    for _ in range(4):
        graph.replay()
        B.attn_weigh(*args[:4], eager, 0.5)
        torch.cuda.synchronize()
        assert torch.equal(acc, eager)


# ---- eviction -----------------------------------------------------------------------------------------

def evict(weights, table, lens, page, budget, sink, recent, **kw):
    dev = device()
    got = B.kv_evict(torch.from_numpy(weights).to(dev), to(dev, table), to(dev, lens), page, budget, sink, recent, **kw)
    want = G.eviction(weights, np.asarray(table), lens, page, budget, sink, recent)
    for g, w, name in zip(got, want, ("table", "lens", "freed", "weights")):
        assert np.array_equal(g.cpu().numpy(), w, equal_nan=True), (name, budget, sink, recent)
    return got


@pytest.mark.parametrize("budget", [1, 2, 5, 8, 12, 13, 40])
@pytest.mark.parametrize("sink,recent", [(0, 1), (1, 2), (4, 3), (100, 1), (0, 100), (3, 10 ** 15)])
def test_eviction(budget, sink, recent):
    """Lengths from 0 past the table, pages gone at the start, middle, end and everywhere."""
    rng = np.random.default_rng(budget)
    page, width, hk = 32, 13, 3
    lens = [0, 1, 32, 33, 400, 416, 10 ** 6, -1, 300, 320]
    table = rng.permutation(len(lens) * width).reshape(len(lens), width)
    table[5, [0, 1, 12]], table[6, [5, 6, 7]], table[8, :], table[9, 2:9] = -1, -5, -1, -1
    weights = rng.exponential(size=(len(lens), hk, width)).astype(np.float32)
    evict(weights, table, lens, page, budget, sink, recent)


@pytest.mark.parametrize("width", [1, 1000, 1024, 1025, 4095, 4096, 4097, 9001])
@pytest.mark.parametrize("hk", [1, 8])
def test_many_pages_to_evict(width, hk):
    rng = np.random.default_rng(width)
    weights = np.exp(2 * rng.standard_normal((3, hk, width))).astype(np.float32)
    table = np.where(rng.random((3, width)) < 0.1, -1, rng.integers(0, 10 ** 6, size=(3, width)))
    for budget in (1, max(1, width // 3), width, width + 5):
        evict(weights, table, [width * 16, width * 16 - 9, width * 8], 16, budget, 2, 3)


def test_ties_nan_and_signs():
    """Equal weights keep the earlier page; NaN ranks first, then the order of numbers; -0 is 0."""
    rng = np.random.default_rng(1)
    width = 300
    weights = rng.choice(np.float32([0.0, -0.0, 1.0, 2.0, -3.0]), size=(4, 1, width))
    weights[1, 0, ::7], weights[2, 0, ::5], weights[2, 0, ::11], weights[3] = np.nan, np.inf, -np.inf, 0.0
    table = rng.permutation(4 * width).reshape(4, width)
    for budget in (2, 50, 130, 299):
        evict(weights, table, [width * 16] * 4, 16, budget, 0, 1)


def test_eviction_outputs_and_calls():
    """Outputs given, prepared, on another stream and captured with lengths and weights that change."""
    dev, rng, page = device(), np.random.default_rng(2), 16
    weights = rng.exponential(size=(5, 2, 5000)).astype(np.float32)
    table, lens = rng.permutation(25000).reshape(5, 5000), [80000, 79999, 100, 0, 40000]
    want = [t.clone() for t in evict(weights, table, lens, page, 777, 1, 2)]
    outs = dict(zip(("table_out", "lens_out", "freed", "weights_out"), (torch.empty_like(t).fill_(3) for t in want)))
    w, t, n = torch.from_numpy(weights).to(dev), to(dev, table), to(dev, lens)
    prepared = B.kv_evict_prepared(w, t, n, page, 777, 1, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (B.kv_evict(w, t, n, page, 777, 1, 2, **outs), prepared(), prepared(), B.kv_evict(w, t, n, page, 777, 1, 2, stream=side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.kv_evict(w, t, n, page, 777, 1, 2)
    for length in (80000, 17, 12432, 12433, 0):
        n[0] = length
        w[0].mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        ref = G.eviction(w.cpu().numpy(), table, n.tolist(), page, 777, 1, 2)
        assert all(np.array_equal(g.cpu().numpy(), r) for g, r in zip(got, ref)), length
