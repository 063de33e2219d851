"""GPU parity: attention of one new token per sequence over the paged cache, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu

FORMATS = [B.NVFP4_KV_BF16, B.NVFP4_KV_E4M3, B.NVFP4_KV_NVFP4]
IDS = ["bf16", "e4m3", "nvfp4"]


class Batch:
    """A cache filled through kv_append, with everything outside the sequences' tokens left as NaN-like garbage."""

    def __init__(self, dev, fmt, lens, hq, hk, d, page, seed=0, scales=(1.0, 1.0), spread=1.0, width=None):
        rng = np.random.default_rng(seed)
        self.fmt, self.lens, self.hq, self.hk, self.d, self.page, self.scales = fmt, list(lens), hq, hk, d, page, scales
        b = len(lens)
        self.width = max([1] + [-(-n // page) for n in lens]) if width is None else width
        pages = b * self.width + 2
        self.cache = B.KvCache(pages, page, hk, d, fmt, *scales, device=dev)
        self.cache.pool.fill_(0xff)          # NaN codes, NaN scales, NaN bf16
        order = rng.permutation(pages)
        table = np.full((b, self.width), 2 ** 31 - 1, np.int64)
        slots, at = [], 0
        for i, n in enumerate(lens):
            for p in range(-(-n // page)):
                table[i, p] = order[at]
                at += 1
            j = np.arange(n)
            slots.append(table[i, j // page] * page + j % page)
        slots = np.concatenate(slots).astype(np.int64) if slots else np.zeros(0, np.int64)
        n = len(slots)
        k = torch.from_numpy((rng.standard_normal((n, hk, d)) * spread).astype(np.float32)).to(torch.bfloat16)
        v = torch.from_numpy(rng.standard_normal((n, hk, d)).astype(np.float32)).to(torch.bfloat16)
        if n:
            B.kv_append(self.cache, k.to(dev), v.to(dev), torch.from_numpy(slots).to(dev))
        self.k, self.v = R.stored(k.float().numpy(), fmt, scales[0]), R.stored(v.float().numpy(), fmt, scales[1])
        self.q = torch.from_numpy(rng.standard_normal((b, hq, d)).astype(np.float32)).to(torch.bfloat16)
        self.table = torch.from_numpy(table.astype(np.int32)).to(dev)
        self.seq = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.dev = dev

    def call(self, **kw):
        return B.attn_decode(self.q.to(self.dev), self.cache, self.table, self.seq, lse=True, **kw)

    def check(self, out, lse, scale=None, window=0, gone=(), what=""):
        """gone: (sequence, page index) pairs that hold nothing."""
        scale = self.d ** -0.5 if scale is None else scale
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        start, g, worst = 0, self.hq // self.hk, 0.0
        for b, n in enumerate(self.lens):
            j = np.arange(max(0, n - window) if window else 0, n)
            j = j[[(b, p) not in gone for p in j // self.page]] if len(j) else j
            for h in range(self.hk):
                rows = slice(h * g, (h + 1) * g)
                o, l, pv, size = R.attend(self.q[b, rows].double().numpy(), self.k[start + j, h], self.v[start + j, h], scale)
                bo, bl = R.attend_bounds(size, len(j), self.d, o, pv, l, self.fmt, self.v[start + j, h])
                empty = np.isneginf(l)
                assert np.array_equal(np.isneginf(lse[b, rows]), empty), (what, b, h)
                err = np.abs(out[b, rows] - o)
                assert (err <= bo).all(), (what, "out", b, h, (err / bo).max())
                errl = np.where(empty, 0, np.abs(np.where(empty, 0, lse[b, rows]) - np.where(empty, 0, l)))
                assert (errl <= bl).all(), (what, "lse", b, h, (errl / bl).max())
                worst = max(worst, (err / bo).max())
            start += n
        return worst


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 100, 127, 128, 129, 255, 257, 1000, 4097])
def test_lengths(fmt, n):
    dev = device()
    x = Batch(dev, fmt, [n], 10, 2, 128, 64, seed=n)
    x.check(*x.call())


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("d", [16, 48, 64, 80, 96, 128, 160, 192, 208, 256])
def test_head_sizes(fmt, d):
    dev = device()
    x = Batch(dev, fmt, [70, 300, 5], 6, 2, d, 32, seed=d)
    x.check(*x.call(), what=d)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 7), (8, 4), (5, 1), (16, 1), (17, 1), (32, 2), (40, 1), (66, 2)])
def test_head_groups(fmt, hq, hk):
    dev = device()
    x = Batch(dev, fmt, [200, 0, 33], hq, hk, 64, 16, seed=hq)
    x.check(*x.call(), what=(hq, hk))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 1024])
def test_page_sizes(fmt, page):
    dev = device()
    x = Batch(dev, fmt, [1, page - 1, page, page + 1, 3 * page + 7, 777], 4, 2, 64, page, seed=page)
    x.check(*x.call(), what=page)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("window", [1, 7, 16, 100, 128, 500, 10 ** 12])
def test_windows(fmt, window):
    dev = device()
    x = Batch(dev, fmt, [1, 0, 99, 128, 513, 2000], 5, 1, 128, 48, seed=window % 97)
    x.check(*x.call(window=window), window=window)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_ragged_batches_and_empty_rows(fmt):
    dev = device()
    rng = np.random.default_rng(3)
    for lens in ([0], [0, 0, 0], [0, 5, 0], list(rng.integers(0, 700, size=67)), [3] * 300, [6000, 1, 1, 1],
                 [0] * 511 + [40]):
        x = Batch(dev, fmt, lens, 4, 2, 64, 32, seed=len(lens))
        x.check(*x.call(), what=len(lens))


def test_large_batch_of_rows():
    """More rows than threads of a workgroup share among them: 2000 short sequences."""
    dev = device()
    rng = np.random.default_rng(4)
    x = Batch(dev, B.NVFP4_KV_NVFP4, list(rng.integers(0, 40, size=2000)), 2, 1, 64, 16)
    x.check(*x.call())


def test_largest_batch():
    """65,536 rows of one token or none, over pages that they share: each row is its token's value."""
    dev = device()
    b, page, pages = 65536, 16, 40
    g = torch.Generator().manual_seed(5)
    cache = B.KvCache(pages, page, 1, 64, B.NVFP4_KV_E4M3, device=dev)
    kv = torch.randn(pages * page, 1, 64, generator=g).to(torch.bfloat16)
    B.kv_append(cache, kv.to(dev), kv.to(dev), torch.arange(pages * page, device=dev))
    table = torch.randint(0, pages, (b, 1), generator=g).to(torch.int32)
    lens = torch.randint(0, 2, (b,), generator=g).to(torch.int32)
    lens[0], lens[-1] = 1, 1
    q = torch.randn(b, 1, 64, generator=g).to(torch.bfloat16)
    out, lse = B.attn_decode(q.to(dev), cache, table.to(dev), lens.to(dev), lse=True)
    stored = torch.from_numpy(R.stored(kv.float().numpy(), B.NVFP4_KV_E4M3))[:, 0]
    mine = stored[table[:, 0].long() * page]
    live = (lens == 1)[:, None]
    assert torch.equal(out[:, 0].cpu(), torch.where(live, mine, 0.0).to(torch.bfloat16))
    score = (q[:, 0].double() * mine.double()).sum(-1, keepdim=True) / 8
    size = (q[:, 0].double() * mine.double()).abs().sum(-1, keepdim=True) / 8
    lse = lse.double().cpu()
    assert torch.isneginf(lse[~live]).all()
    # 64 products, one product with the scale, the exponential's, the logarithm's and the sum's own rounding.
    assert ((lse - score).abs() <= (80 * size + 16) * 2.0 ** -24)[live].all()


@pytest.mark.parametrize("hq,hk,d", [(32768, 1, 16), (1024, 1024, 64), (32768, 1024, 16)])
def test_most_heads(hq, hk, d):
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [50], hq, hk, d, 16, seed=hk)
    x.check(*x.call(), what=(hq, hk))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_long_sequence_split_over_every_workgroup(fmt):
    dev = device()
    x = Batch(dev, fmt, [70_001], 2, 1, 64, 256)
    x.check(*x.call())


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_sharp_flat_and_growing_scores(fmt):
    """Scores far apart, all equal, and rising along the sequence (the reference moves at every step)."""
    dev = device()
    x = Batch(dev, fmt, [900], 5, 1, 128, 64, seed=1, spread=20.0)
    x.check(*x.call(), what="sharp")
    x.check(*x.call(scale=1e-6), scale=1e-6, what="flat")
    for sign in (1, -1):
        y = Batch(dev, fmt, [900], 5, 1, 128, 64, seed=2)
        ramp = torch.arange(1, 901, dtype=torch.float32)[:, None, None] * 0.05 * sign
        k = (ramp.expand(900, 1, 128) * 0.5).to(torch.bfloat16)
        v = torch.randn(900, 1, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        slots = (y.table[0].long()[torch.arange(900, device=dev) // 64] * 64 + torch.arange(900, device=dev) % 64)
        B.kv_append(y.cache, k.to(dev), v.to(dev), slots)
        y.k, y.v = R.stored(k.float().numpy(), fmt), R.stored(v.float().numpy(), fmt)
        y.q = torch.ones(1, 5, 128, dtype=torch.bfloat16)
        y.check(*y.call(), what=sign)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("shift", [0, 24, 26, 28, 32, 90])
def test_scores_far_beyond_the_exponentials_range(fmt, shift):
    """Scores of +-2^shift times small integers, exact in fp32: at 2^24 all weight is on the largest, however far
    below zero, and equal ones share it.  log2 e enters once, rounded, so the lse is off relative to its size."""
    dev = device()
    n, page = 700, 64
    x = Batch(dev, fmt, [n, n], 2, 1, 64, page)
    c = torch.arange(2 * n) % 5 + 2                       # 2 .. 6: E2M1 and E4M3 values times a power of two
    c[c == 5] = 4
    k = torch.zeros(2 * n, 1, 64)
    k[:, 0, 0] = c
    v = torch.randn(2 * n, 1, 64, generator=torch.Generator().manual_seed(shift)).to(torch.bfloat16)
    at = torch.arange(2 * n)
    slots = x.table.cpu().long()[at // n, at % n // page] * page + at % n % page
    B.kv_append(x.cache, k.to(torch.bfloat16).to(dev), v.to(dev), slots.to(dev))
    x.k, x.v = R.stored(k.numpy(), fmt), R.stored(v.float().numpy(), fmt)
    x.q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    x.q[0, 0, 0], x.q[0, 1, 0], x.q[1, 0, 0], x.q[1, 1, 0] = 1.0, -1.0, -0.75, 2.0
    if shift == 0:
        x.check(*x.call(scale=1.0), scale=1.0)
        return
    out, lse = x.call(scale=2.0 ** shift)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(2):
        for h in range(2):
            s = float(x.q[b, h, 0]) * x.k[b * n:(b + 1) * n, 0, 0] * 2.0 ** shift
            rows = x.v[b * n:(b + 1) * n, 0][s == s.max()]
            o = rows.mean(0)
            # As many equal terms, a sum and a quotient in fp32, and one rounding to bf16.
            bound = 2.0 ** -8 * np.abs(o) + (len(rows) + 8) * 2.0 ** -24 * np.abs(rows).mean(0) + 1e-30
            if fmt == B.NVFP4_KV_NVFP4:
                bound += 2.0 ** -11 * np.abs(rows).mean(0)
            assert (np.abs(out[b, h] - o) <= bound).all(), (b, h)
            assert abs(lse[b, h] - s.max()) <= 2.0 ** -20 * abs(s.max())


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("gap", [10, 20, 25, 28, 31, 34, 36, 40, 60])
def test_terms_far_below_the_largest(fmt, gap):
    """A token at the maximum whose values are zero, and some 2^-gap of it or less that make up the whole output."""
    dev = device()
    x = Batch(dev, fmt, [40], 1, 1, 64, 64)
    k, v = torch.zeros(40, 1, 64), torch.randn(40, 1, 64, generator=torch.Generator().manual_seed(gap)).to(torch.bfloat16)
    k[7, 0, 0], k[30:, 0, 0] = 6.0, -0.5
    v[7] = 0.0
    slots = (x.table[0].long()[torch.arange(40, device=dev) // 64] * 64 + torch.arange(40, device=dev) % 64)
    B.kv_append(x.cache, k.to(torch.bfloat16).to(dev), v.to(dev), slots)
    x.k, x.v = R.stored(k.numpy(), fmt), R.stored(v.float().numpy(), fmt)
    x.q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    x.q[0, 0, 0] = 1.0
    scale = gap * np.log(2) / 6
    x.check(*x.call(scale=scale), scale=scale)


def test_small_terms_add_up():
    """One token at the maximum and 60,000 that each weigh 2^-20 of it: no term may be lost to a 16-bit range."""
    dev = device()
    n = 60_000
    for fmt in FORMATS:
        x = Batch(dev, fmt, [n], 1, 1, 64, 256)
        k = torch.zeros(n, 1, 64)
        k[n // 3, 0, 0] = 6.0
        v = torch.ones(n, 1, 64)
        v[n // 3] = -1.0
        slots = (x.table[0].long()[torch.arange(n, device=dev) // 256] * 256 + torch.arange(n, device=dev) % 256)
        B.kv_append(x.cache, k.to(dev), v.to(dev), slots)
        x.k, x.v = R.stored(k.numpy(), fmt), R.stored(v.numpy(), fmt)
        x.q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
        x.q[0, 0, 0] = 1.0
        scale = 20 * np.log(2) / 6
        x.check(*x.call(scale=scale), scale=scale, what=fmt)


def test_tensor_scales_and_query_range():
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [333, 20], 6, 2, 128, 64, scales=(0.25, 3.0))
    x.check(*x.call())
    x = Batch(dev, B.NVFP4_KV_NVFP4, [333, 20], 6, 2, 128, 64, scales=(2.0 ** -40, 2.0 ** 30))
    for size in (2.0 ** -60, 2.0 ** 40):
        y = Batch(dev, B.NVFP4_KV_NVFP4, [333, 20], 6, 2, 128, 64, scales=(1.0, 1.0))
        y.q = (y.q.float() * size).to(torch.bfloat16)
        scale = 1 / (size * 11)
        y.check(*y.call(scale=scale), scale=scale, what=size)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_evicted_pages(fmt):
    """Page ids outside the pool hold nothing; a row whose pages are all gone is empty."""
    dev = device()
    x = Batch(dev, fmt, [300, 300, 90], 4, 2, 64, 48, seed=9)
    gone = [(0, 0), (0, 3), (1, 6), (2, 0), (2, 1)]
    for b, p in gone:
        x.table[b, p] = [-1, 10 ** 9, x.cache.pages, -2 ** 31, -7][(b + p) % 5]
    x.check(*x.call(), gone=set(gone))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_lengths_out_of_range(fmt):
    """Negative lengths count as 0, lengths past the table as the table's."""
    dev = device()
    x = Batch(dev, fmt, [96, 96, 0], 4, 2, 64, 48, seed=2)
    x.seq = torch.tensor([10 ** 9, 96, -5], dtype=torch.int32, device=dev)
    x.check(*x.call())


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_nan_in_a_row_stays_in_its_head(fmt):
    dev = device()
    x = Batch(dev, fmt, [200, 50], 4, 2, 64, 32, seed=1)
    bad = torch.ones(1, 2, 64, device=dev)
    bad[0, 1, 5] = float("nan")
    slot = (x.table[0, 1].long() * 32 + 3).view(1)
    for side in (0, 1):
        y = Batch(dev, fmt, [200, 50], 4, 2, 64, 32, seed=1)
        ok = torch.ones(1, 2, 64, device=dev)
        B.kv_append(y.cache, *((bad, ok) if side == 0 else (ok, bad)), slot)
        out, lse = y.call()
        assert not out[0, :2].isnan().any() and not out[1].isnan().any() and not lse[1].isnan().any()
        assert out[0, 2:].isnan().any(-1).all()
        assert lse[0, 2:].isnan().all() == (side == 0)


def test_strided_rows_and_untouched_neighbours():
    dev = device()
    x = Batch(dev, B.NVFP4_KV_E4M3, [100, 64, 7], 4, 2, 80, 32, seed=2)
    wide_q = torch.full((3, 4 * 80 + 64), float("nan"), dtype=torch.bfloat16, device=dev)
    q = wide_q[:, :320].unflatten(1, (4, 80))
    q.copy_(x.q)
    wide_o = torch.full((4, 4 * 80 + 40), 9.0, dtype=torch.bfloat16, device=dev)
    out = wide_o[:3, :320].unflatten(1, (4, 80))
    lse = torch.empty(3, 4, device=dev)
    B.attn_decode(q, x.cache, x.table, x.seq, out=out, lse=lse)
    x.check(out, lse)
    assert (wide_o[:, 320:] == 9.0).all() and (wide_o[3] == 9.0).all()


def test_repeats_are_bit_identical_and_leave_counters_zero():
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [5000, 30, 1200], 10, 2, 128, 64, seed=2)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    first = x.call(ws=ws)
    for _ in range(5):
        again = x.call(ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    y = Batch(dev, B.NVFP4_KV_BF16, [3000] * 3, 4, 1, 256, 64, seed=2)     # another shape through the same workspace
    y.check(*y.call(ws=ws))
    assert not ws[:1024].any()
    assert torch.equal(first[0], x.call(ws=ws)[0])


def test_capture_and_replay():
    """A captured call replayed among eager calls on the same stream, over changing lengths and queries."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [2000, 700, 1], 10, 2, 128, 64, seed=2)
    q, seq = x.q.to(dev), x.seq.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        B.attn_decode(q, x.cache, x.table, seq, lse=True)
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = B.attn_decode(q, x.cache, x.table, seq, lse=True)
            graphs.append((g, out))
    torch.cuda.synchronize()
    for step, lens in enumerate(([2000, 700, 1], [1, 0, 1], [1999, 333, 0], [2000, 700, 1])):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        x.seq.copy_(seq)
        q.mul_(-1 if step % 2 else 1)
        want = B.attn_decode(q, x.cache, x.table, seq, lse=True)
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = B.attn_decode(q, x.cache, x.table, seq, lse=True)
        torch.cuda.synchronize()
        for g, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), step
        assert torch.equal(eager[0], want[0])


def test_streams_overlap():
    """Calls on several streams, each with its own default workspace; and a call told its stream."""
    dev = device()
    xs = [Batch(dev, f, [3000, 100], 10, 2, 128, 64, seed=s) for s, f in enumerate(FORMATS)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(10):
        got = []
        for x, s in zip(xs, streams):
            q = x.q.to(dev)
            s.wait_stream(torch.cuda.current_stream())
            got.append(B.attn_decode(q, x.cache, x.table, x.seq, lse=True, stream=s))
            q.record_stream(s)
    torch.cuda.synchronize()
    for x, o in zip(xs, got):
        x.check(*o)


def test_prepared_call():
    dev = device()
    x = Batch(dev, B.NVFP4_KV_E4M3, [500, 64], 8, 2, 64, 32)
    call = B.attn_decode_prepared(x.q.to(dev), x.cache, x.table, x.seq, lse=True)
    a = [t.clone() for t in call()]
    b = call()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x.check(*b)


def test_shared_pages_as_several_new_tokens():
    """Three new tokens of one sequence as rows with the same table and lengths n, n + 1, n + 2."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [402], 5, 1, 128, 64, seed=4)
    q = torch.randn(3, 5, 128, device=dev).to(torch.bfloat16)
    lens = torch.tensor([400, 401, 402], dtype=torch.int32, device=dev)
    out, lse = B.attn_decode(q, x.cache, x.table.expand(3, -1).contiguous(), lens, lse=True)
    for i in range(3):
        y = Batch.__new__(Batch)
        y.__dict__.update(x.__dict__)
        y.lens, y.q = [400 + i], q[i:i + 1].cpu()
        y.check(out[i:i + 1], lse[i:i + 1])


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_offsets_past_32_bits(fmt):
    """Groups, slots and scales whose byte offsets in the pool pass 2^32: pages at both ends of a large pool."""
    dev = device()
    page, hk, d = 64, 8, 128
    group = {0: 8192, 1: 4128, 2: 2304}[fmt]
    pages = (5 << 30) // (group * hk * page // 16)
    cache = B.KvCache(pages, page, hk, d, fmt, device=dev)
    assert cache.pool.numel() > 1 << 32
    g = torch.Generator().manual_seed(1)
    ids = torch.tensor([[pages - 1, 0, pages // 2, pages - 2]], dtype=torch.int32)
    n = 4 * page - 5
    j = torch.arange(n)
    slots = ids[0].long()[j // page] * page + j % page
    k, v = (torch.randn(n, hk, d, generator=g).to(torch.bfloat16) for _ in range(2))
    B.kv_append(cache, k.to(dev), v.to(dev), slots.to(dev))
    k2, v2 = B.kv_read(cache, slots.to(dev), dtype=torch.float32)
    ks, vs = R.stored(k.float().numpy(), fmt), R.stored(v.float().numpy(), fmt)
    assert np.array_equal(k2.double().cpu().numpy(), ks) and np.array_equal(v2.double().cpu().numpy(), vs)
    x = Batch.__new__(Batch)
    x.fmt, x.lens, x.hq, x.hk, x.d, x.page, x.k, x.v = fmt, [n], 2 * hk, hk, d, page, ks, vs
    x.q = torch.randn(1, 2 * hk, d, generator=g).to(torch.bfloat16)
    out, lse = B.attn_decode(x.q.to(dev), cache, ids.to(dev), torch.tensor([n], dtype=torch.int32, device=dev), lse=True)
    x.check(out, lse)
