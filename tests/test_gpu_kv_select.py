"""GPU parity: page bounds, selection by them and attention over pages of each kv head's own, against the definitions."""
import numpy as np
import pytest
import torch

import long_reference as G
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu


def to(dev, a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device=dev)


# ---- bounds ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("d", [16, 48, 64, 80, 96, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("page", [16, 32, 48, 80])
def test_bounds(fmt, d, page):
    """Exact, whatever the tensor scale; unlisted pages stay as they were, ids outside the pool are skipped."""
    dev = device()
    scales = (0.0371, 2.0) if fmt == B.NVFP4_KV_NVFP4 else (1.0, 1.0)
    pool = G.Pool(dev, fmt, 7, page, 3, d, seed=d + page, scales=scales)
    bounds = torch.full((7, 3, 2, d), 5.0, dtype=torch.bfloat16, device=dev)
    got = B.kv_bounds(pool.cache, to(dev, [6, 0, -1, 3, 7, 3, 2 ** 31 - 1, 4]), bounds)
    assert got is bounds
    # (The tests' reference has the tensor scale in its values: taken out again, to the nearest bf16 number.)
    want = torch.from_numpy(pool.bounds()).to(torch.bfloat16).double()
    listed = [0, 3, 4, 6]
    assert torch.equal(bounds.double().cpu()[listed], want[listed])
    assert (bounds[[1, 2, 5]] == 5.0).all()
    assert B.kv_bounds(pool.cache, to(dev, [])).shape == (7, 3, 2, d)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
def test_bounds_of_infinities_and_nan(fmt):
    """A channel with a NaN (E4M3: the row, NVFP4: the block) has NaN in both bounds, the others theirs."""
    dev, d, page = device(), 64, 16
    pool = G.Pool(dev, fmt, 4, page, 1, d, seed=2)
    k = torch.randn(2, 1, d).to(torch.bfloat16)
    k[0, 0, 5], k[1, 0, 40] = float("nan"), float("-inf")
    pool.write([3, 2 * page + 7], k, torch.zeros(2, 1, d, dtype=torch.bfloat16))
    got = B.kv_bounds(pool.cache, to(dev, [0, 1, 2, 3])).double().cpu().numpy()
    want = pool.bounds()
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got[0, 0, :, 5]).all() and not np.isnan(got[1]).any()
    if fmt == B.NVFP4_KV_BF16:
        assert got[2, 0, 0, 40] == -np.inf and np.isnan(got).sum() == 2


def test_bounds_of_signs_and_zeros():
    """All of one sign, zeros of both signs, subnormal numbers and the largest."""
    dev, d, page = device(), 16, 16
    pool = G.Pool(dev, B.NVFP4_KV_BF16, 2, page, 1, d, seed=3)
    k = torch.zeros(page, 1, d, dtype=torch.bfloat16)
    k[:, 0, 0] = torch.linspace(1, 2, page)
    k[:, 0, 1] = -torch.linspace(1, 2, page)
    k[::2, 0, 2] = -0.0
    k[:, 0, 3] = torch.tensor([(-1) ** i * i * 2.0 ** -133 for i in range(page)])
    k[:, 0, 4] = torch.finfo(torch.bfloat16).max
    k[3, 0, 5] = torch.finfo(torch.bfloat16).min
    pool.write(np.arange(page), k, k)
    got = B.kv_bounds(pool.cache, to(dev, [0])).double().cpu().numpy()[0]
    assert np.array_equal(got, pool.bounds()[0])


# ---- selection ---------------------------------------------------------------------------------------

def select(pool, q, table, lens, budget, bounds=None, **kw):
    dev = pool.dev
    bounds = B.kv_bounds(pool.cache, to(dev, np.arange(pool.pages))) if bounds is None else bounds
    pages, tokens = B.kv_select(q.to(dev), pool.cache, bounds, to(dev, table), to(dev, lens), budget, **kw)
    return pages.cpu().numpy(), tokens.cpu().numpy(), bounds.double().cpu().numpy()


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("budget", [1, 2, 3, 7, 20, 21, 64])
def test_selection_and_attention(fmt, budget):
    """Ragged lengths from nothing on, pages that are gone, tables that two sequences share; then attention over them."""
    dev, page, hk, d, hq = device(), 16, 3, 64, 6
    rng = np.random.default_rng(budget)
    pool = G.Pool(dev, fmt, 90, page, hk, d, seed=budget, around=1.0)
    lens = [0, 1, 16, 17, 330, 335, 200, -3, 10 ** 6]
    table = np.stack([rng.permutation(90)[:21] for _ in lens])
    table[4, [0, 5]], table[5, 20], table[6, :] = -1, 90, table[5, :]
    q = G.queries(len(lens), hq, d, seed=3, spread=2.0)
    pages, tokens, bounds = select(pool, q, table, lens, budget)
    want, want_tokens = G.selection(q, bounds, table, lens, budget, page, 90)
    assert np.array_equal(tokens, want_tokens)
    assert np.array_equal(pages, want)
    out, lse = B.attn_decode(q.to(dev), pool.cache, to(dev, pages), to(dev, tokens), lse=True)
    lists = [[pool.slots(pages[b, h], tokens[b])[0] for h in range(hk)] for b in range(len(lens))]
    G.check_rows(pool, q, lists, out, lse)


@pytest.mark.parametrize("d", [16, 48, 80, 96, 128, 160, 192, 208, 256])
@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 1), (16, 2), (17, 1), (40, 1), (24, 8)])
def test_head_sizes_and_groups(d, hq, hk):
    dev, page = device(), 16
    rng = np.random.default_rng(d)
    pool = G.Pool(dev, B.NVFP4_KV_NVFP4, 40, page, hk, d, seed=d, around=0.5, scales=(0.11, 1.0))
    lens, table = [16 * 33 - 5, 16 * 30], np.stack([rng.permutation(40)[:33] for _ in range(2)])
    q = G.queries(2, hq, d, seed=d)
    pages, tokens, bounds = select(pool, q, table, lens, 9)
    want, want_tokens = G.selection(q, bounds, table, lens, 9, page, 40)
    assert np.array_equal(pages, want) and np.array_equal(tokens, want_tokens)


def random_bounds(rng, pages, hk, d):
    b = np.sort(rng.standard_normal((pages, hk, 2, d)), axis=2)
    return torch.from_numpy(b.astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("n", [65, 100, 1000, 4095, 4096, 4097, 4098, 9000])
@pytest.mark.parametrize("users,hk", [(1, 1), (2, 5), (150, 8)])
def test_many_pages(n, users, hk):
    """Scores cut over workgroups, in LDS and in memory, and whole tables a workgroup (1200 pairs)."""
    if users == 150 and n > 4098:
        n = 4097 + 500
    dev, d, page, pages = device(), 16, 16, 2000
    rng = np.random.default_rng(n)
    cache = B.KvCache(pages, page, hk, d, B.NVFP4_KV_BF16, device=dev)
    bounds = random_bounds(rng, pages, hk, d)
    table = rng.integers(0, pages, size=(users, n))
    lens = np.full(users, n * page)
    lens[users // 2:] -= rng.integers(0, n * page, size=users - users // 2)
    q = G.queries(users, 2 * hk, d, seed=n)
    for budget in (2, 33, n // 2, n - 1):
        got, tokens = B.kv_select(q.to(dev), cache, bounds.to(dev), to(dev, table), to(dev, lens), budget)
        got = got.cpu().numpy()
        some = range(users) if users < 3 else [0, 77, users - 1]
        want, want_tokens = G.selection(q[list(some)], bounds.double().numpy(), table[list(some)], lens[list(some)], budget, page, pages)
        assert np.array_equal(got[list(some)], want), (n, users, budget)
        assert np.array_equal(tokens.cpu().numpy()[list(some)], want_tokens)


@pytest.mark.parametrize("n,users", [(50, 3), (3000, 1), (5000, 2)])
def test_ties_go_to_the_earlier_page(n, users):
    """Few distinct pages, each listed over and over: scores that are equal to the last bit, -0 and +0 among them."""
    dev, d, page, pages, hk = device(), 32, 16, 5, 2
    rng = np.random.default_rng(n)
    cache = B.KvCache(pages, page, hk, d, B.NVFP4_KV_BF16, device=dev)
    bounds = random_bounds(rng, pages, hk, d)
    bounds[3], bounds[4] = 0.0, -0.0
    table = rng.integers(0, pages, size=(users, n))
    lens = np.full(users, n * page - 3)
    q = G.queries(users, 2 * hk, d, seed=n)
    for budget in (2, 10, n // 3, n // 2, n - 1):
        got, _ = B.kv_select(q.to(dev), cache, bounds.to(dev), to(dev, table), to(dev, lens), budget)
        want, _ = G.selection(q, bounds.double().numpy(), table, lens, budget, page, pages)
        assert np.array_equal(got.cpu().numpy(), want), (n, budget)
    zero = torch.zeros_like(q)
    got, _ = B.kv_select(zero.to(dev), cache, bounds.to(dev), to(dev, table), to(dev, lens), 7)
    assert np.array_equal(got.cpu().numpy()[:, 0, :6], table[:, :6])


def test_infinite_and_nan_scores():
    """NaN first, then +inf, the rest by size, -inf before pages that are not there; far exponents are not lost."""
    dev, d, page, pages = device(), 16, 16, 8
    cache = B.KvCache(pages, page, 1, d, B.NVFP4_KV_BF16, device=dev)
    bounds = torch.zeros(pages, 1, 2, d, dtype=torch.bfloat16)
    bounds[0, 0, :, 0], bounds[1, 0, :, 0], bounds[2, 0, :, 0] = float("nan"), float("inf"), float("-inf")
    bounds[3, 0, :, 0], bounds[4, 0, :, 0], bounds[5, 0, :, 0] = 3e38, 1e-38, -3e38
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16)
    q[..., 0], q[..., 1:] = 3e38, 1.0
    table = to(dev, [[2, 7, 5, -1, 4, 3, 1, 0, 6]])
    lens = to(dev, [9 * page])
    orders = {1: [], 2: [0], 3: [1, 0], 4: [3, 1, 0], 5: [4, 3, 1, 0], 6: [7, 4, 3, 1, 0], 7: [7, 5, 4, 3, 1, 0],
              8: [2, 7, 5, 4, 3, 1, 0], 9: [2, 7, 5, 4, 3, 1, 0]}
    for budget, want in orders.items():
        got, tokens = B.kv_select(q.to(dev), cache, bounds.to(dev), table, lens, budget)
        assert got.cpu().tolist() == [[want + [6] + [-1] * (budget - 1 - len(want))]], budget
        assert tokens.item() == (len(want) + 1) * page
    # Products of 2^-133 by 2^-133 still tell pages apart.
    bounds.zero_()
    bounds[0, 0, :, 0], bounds[1, 0, :, 0] = 2.0 ** -133, 2.0 ** -132
    got, _ = B.kv_select(torch.full_like(q, 2.0 ** -133).to(dev), cache, bounds.to(dev), to(dev, [[0, 2, 1, 3]]), to(dev, [64]), 2)
    assert got.cpu().tolist() == [[[1, 3]]]


@pytest.mark.parametrize("d", [16, 128, 192, 256])
@pytest.mark.parametrize("rows", [1, 5, 20])
def test_bounds_that_are_not_finite_beside_others(d, rows):
    """Infinities on the side that a query's sign does not ask for do not count (zeros ask for hi), those on the other do."""
    dev, page, pages, n = device(), 16, 300, 200
    rng = np.random.default_rng(d + rows)
    cache = B.KvCache(pages, page, 1, d, B.NVFP4_KV_BF16, device=dev)
    bounds = random_bounds(rng, pages, 1, d)
    q = G.queries(2, rows, d, seed=d)
    q[:, :, 3], q[:, :, 4], q[:, :, 5], q[:, :, 6] = 1.0, -1.0, 0.0, -0.0
    inf = float("inf")
    for p, (channel, side, value) in zip(range(0, 300, 7), [(c, s, v) for c in (3, 4, 5, 6) for s in (0, 1) for v in (inf, -inf, float("nan"))]):
        bounds[p, 0, side, channel] = value
    table = np.stack([rng.permutation(pages)[:n] for _ in range(2)])
    lens = [n * page, 150 * page + 3]
    for budget in (2, 9, 30, 150):
        got, tokens = B.kv_select(q.to(dev), cache, bounds.to(dev), to(dev, table), to(dev, lens), budget)
        with np.errstate(invalid="ignore"):
            want, want_tokens = G.selection(q, bounds.double().numpy(), table, lens, budget, page, pages)
        assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(tokens.cpu().numpy(), want_tokens), budget


def test_calls_of_all_kinds():
    """Repeated, prepared, on another stream, captured with lengths that change, outputs given, workspaces shared: same results,
    counters left zero."""
    dev, d, page, pages, hk = device(), 64, 16, 600, 2
    rng = np.random.default_rng(5)
    cache = B.KvCache(pages, page, hk, d, B.NVFP4_KV_BF16, device=dev)
    bounds = random_bounds(rng, pages, hk, d)
    table = np.stack([rng.permutation(pages)[:500] for _ in range(3)])
    lens = np.array([500 * page, 3000, 20])
    q = G.queries(3, 6, d)
    args = [q.to(dev), cache, bounds.to(dev), to(dev, table), to(dev, lens), 30]
    want = [torch.as_tensor(t).int() for t in G.selection(q, bounds.double().numpy(), table, lens, 30, page, pages)]
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=dev)
    out = (torch.full((3, hk, 30), 7, dtype=torch.int32, device=dev), torch.full((3,), 7, dtype=torch.int32, device=dev))
    prepared = B.kv_select_prepared(*args)
    assert prepared.outputs[0].shape == (3, hk, 30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for got in (B.kv_select(*args), prepared(), B.kv_select(*args, pages_out=out[0], lens_out=out[1], ws=ws),
                    B.kv_select(*args, stream=side)):
            torch.cuda.synchronize()
            assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
        assert (ws[:B.NVFP4_SELECT_COUNTER_BYTES] == 0).all()
        # Another shape on the same workspace, whose counters and keys lie elsewhere.
        B.kv_select(args[0][:1], cache, args[2], args[3][:1], args[4][:1], 3, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.kv_select(*args)
        o = B.attn_decode(args[0], cache, got[0], got[1])
    for n in (500 * page, 481, 480, 0, 7777):
        args[4][0] = n
        lens[0] = n
        got[0].fill_(99)
        graph.replay()
        eager = B.kv_select(*args)
        torch.cuda.synchronize()
        want = G.selection(q, bounds.double().numpy(), table, lens, 30, page, pages)
        for e, c, w in zip(eager, got, want):
            assert np.array_equal(c.cpu().numpy(), w) and torch.equal(e, c), n
    assert o.shape == (3, 6, d)


# ---- attention with a page table for each kv head ---------------------------------------------------

@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("hq,hk", [(3, 3), (20, 4), (34, 2)])
def test_tables_of_each_head(fmt, d, hq, hk):
    """Tables that differ from head to head, evicted pages in some, lengths from 0 on, a window."""
    dev, page = device(), 32
    rng = np.random.default_rng(d + hq)
    pool = G.Pool(dev, fmt, 30, page, hk, d, seed=d)
    lens = [0, 1, 100, 32 * 12, 333]
    table = rng.integers(0, 30, size=(len(lens), hk, 12))
    table[3, 0, 4], table[3, 1, :], table[4, hk - 1, 10] = -1, -1, 30
    q = G.queries(len(lens), hq, d, seed=d)
    for window in (0, 50):
        out, lse = B.attn_decode(q.to(dev), pool.cache, to(dev, table), to(dev, lens), lse=True, window=window)
        lists = [[pool.slots(table[b, h], n, max(0, n - window) if window else 0)[0] for h in range(hk)] for b, n in enumerate(lens)]
        G.check_rows(pool, q, lists, out, lse, what=window)
    call = B.attn_decode_prepared(q.to(dev), pool.cache, to(dev, table), to(dev, lens), lse=True, window=50)
    assert all(torch.equal(a, b) for a, b in zip(call(), (out, lse)))
