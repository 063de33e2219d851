"""Reading less of a long cache, from the definitions, on the CPU in 64 bits (no code shared with the library)."""
import numpy as np
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B

FORMATS = [B.NVFP4_KV_BF16, B.NVFP4_KV_E4M3, B.NVFP4_KV_NVFP4]
IDS = ["bf16", "e4m3", "nvfp4"]


class Pool:
    """A cache whose listed pages (default: all) are written, with garbage (NaN codes and scales) elsewhere.  k and v hold
    what the cache stands for, [slots][heads][d], NaN where nothing was written."""

    def __init__(self, dev, fmt, pages, page, hk, d, seed=0, scales=(1.0, 1.0), spread=1.0, slots=None, around=0.0):
        rng = np.random.default_rng(seed)
        self.dev, self.fmt, self.pages, self.page, self.hk, self.d, self.scales = dev, fmt, pages, page, hk, d, scales
        self.cache = B.KvCache(pages, page, hk, d, fmt, *scales, device=dev)
        self.cache.pool.fill_(0xff)
        slots = np.arange(pages * page) if slots is None else np.asarray(slots, np.int64)
        n = len(slots)
        k = rng.standard_normal((n, hk, d)) * spread
        if around:                      # keys of one page lie around a direction of their own
            k += (rng.standard_normal((pages, hk, d)) * around)[slots // page]
        k = torch.from_numpy(k.astype(np.float32)).to(torch.bfloat16)
        v = torch.from_numpy(rng.standard_normal((n, hk, d)).astype(np.float32)).to(torch.bfloat16)
        self.k, self.v = (np.full((pages * page, hk, d), np.nan) for _ in range(2))
        self.write(slots, k, v)

    def write(self, slots, k, v):
        if len(slots):
            B.kv_append(self.cache, k.to(self.dev), v.to(self.dev), torch.from_numpy(np.asarray(slots, np.int64)).to(self.dev))
            self.k[slots] = R.stored(k.float().numpy(), self.fmt, self.scales[0])
            self.v[slots] = R.stored(v.float().numpy(), self.fmt, self.scales[1])

    def slots(self, table, n, first=0):
        """The slots of tokens first .. n - 1 of a page table (ids outside the pool hold nothing), and their places."""
        j = np.arange(first, max(first, min(n, len(table) * self.page)))
        page = np.asarray(table, np.int64)[j // self.page]
        there = (page >= 0) & (page < self.pages)
        return (page * self.page + j % self.page)[there], j[there]

    def bounds(self):
        k = (self.k / self.scales[0]).reshape(self.pages, self.page, self.hk, self.d)
        return np.stack((k.min(1), k.max(1)), 2)


def with_room(prefix_pages, fmt, batch, hq, hk, d, page):
    """A prefix's table with places for so many more pages (ids that hold nothing) that its tokens are read for all sequences at
    once, not by each: beyond 96 MB of codes."""
    group = 16 * 2 * 64 * -(-d // 64) * {0: 4, 1: 2, 2: 1}[fmt] // 2
    each = batch * -(-hq // hk // 16) * hk * (page // 16) * group
    return np.concatenate((prefix_pages, np.full((97 << 20) // each + 1, 2 ** 31 - 1))).astype(np.int32)


def queries(b, hq, d, seed=1, spread=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal((b, hq, d)) * spread).astype(np.float32)).to(torch.bfloat16)


def check_rows(pool, q, lists, out, lse, scale=None, what=""):
    """out and lse of rows that attend to lists[b], or lists[b][h] for a list of each kv head: slots."""
    scale = pool.d ** -0.5 if scale is None else scale
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    g = q.shape[1] // pool.hk
    for b in range(q.shape[0]):
        for h in range(pool.hk):
            rows = slice(h * g, (h + 1) * g)
            at = lists[b][h] if isinstance(lists[b], list) else lists[b]
            k, v = pool.k[at, h], pool.v[at, h]
            o, l, pv, size = R.attend(q[b, rows].double().numpy(), k, v, scale)
            bo, bl = R.attend_bounds(size, len(at), pool.d, o, pv, l, pool.fmt, v)
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[b, rows]), empty), (what, b, h, lse[b, rows])
            err = np.abs(out[b, rows] - o)
            assert (err <= bo).all(), (what, "out", b, h, np.nanmax(err / bo))
            errl = np.where(empty, 0, np.abs(np.where(empty, 0, lse[b, rows]) - np.where(empty, 0, l)))
            assert (errl <= bl).all(), (what, "lse", b, h, np.nanmax(errl / bl))


def page_weights(pool, q, table, lens, width, scale=None, window=0):
    """(sum over a kv head's rows of each page's terms [b][hk][width], how far fp32 sums may be off).

    A term exp(s - lse): the score is off by (d + 4) half steps of sum |q k|, lse by its own bound (R.attend_bounds).  The
    sum of sixteen terms is kept as a logarithm with the reference in it: half a step of at most log2 e (|s| + 1), carried
    through the exponential, and half a step each for lse's product and the difference; the two exponentials and the logarithm
    take four half steps each; sums of n terms n half steps."""
    scale = pool.d ** -0.5 if scale is None else scale
    g = q.shape[1] // pool.hk
    w, off = np.zeros((q.shape[0], pool.hk, width)), np.zeros((q.shape[0], pool.hk, width))
    for b in range(q.shape[0]):
        n = min(lens[b], width * pool.page)
        at, j = pool.slots(table[b], n, max(0, n - window) if window else 0)
        for h in range(pool.hk):
            qh, k, v = q[b, h * g:(h + 1) * g].double().numpy(), pool.k[at, h], pool.v[at, h]
            if not len(at):
                continue
            o, l, pv, size = R.attend(qh, k, v, scale)
            _, bl = R.attend_bounds(size, len(at), pool.d, o, pv, l, pool.fmt, v)
            p = np.exp(qh @ k.T * scale - l[:, None])
            rel = (pool.d + 4) * R.U24 * size + bl + R.U24 * (12 + 3 * 2 * (size + np.abs(l) + 1) + 16 + g * (pool.page // 16 + 2))
            for r in range(g):
                np.add.at(w[b, h], j // pool.page, p[r])
                np.add.at(off[b, h], j // pool.page, p[r] * rel[r])
    return w, off + 1e-30


def selection(q, bounds, table, lens, budget, page, pages):
    """(pages [b][hk][budget], lens [b]) by the definition, scores in long double."""
    b, hk = q.shape[0], bounds.shape[1]
    g = q.shape[1] // hk
    out, tokens = np.full((b, hk, budget), -1, np.int64), np.zeros(b, np.int64)
    for i in range(b):
        n = min(max(int(lens[i]), 0), table.shape[1] * page)
        blocks = -(-n // page)
        if not blocks:
            continue
        there = [j for j in range(blocks - 1) if 0 <= table[i, j] < pages]
        for h in range(hk):
            qh = q[i, h * g:(h + 1) * g].double().numpy().astype(np.longdouble)
            score = {}
            for j in there:
                lo, hi = bounds[table[i, j], h].astype(np.longdouble)
                s = np.where(qh < 0, qh * lo, qh * hi).sum(-1)
                score[j] = (0, 0.0) if np.isnan(s).any() else (1, -float(s.max()))   # a NaN above everything
            best = sorted(sorted(there, key=lambda j: (*score[j], j))[:budget - 1])
            chosen = [table[i, j] for j in best] + [table[i, blocks - 1] if 0 <= table[i, blocks - 1] < pages else -1]
            out[i, h, :len(chosen)] = chosen
            tokens[i] = (len(chosen) - 1) * page + (n - 1) % page + 1
    return out, tokens


def eviction(weights, table, lens, page, budget, sink, recent):
    """(table, lens, freed, weights) by the definition."""
    b, hk, width = weights.shape
    out, tokens = np.full((b, budget), -1, np.int64), np.zeros(b, np.int64)
    freed, moved = np.full((b, width), -1, np.int64), np.zeros((b, hk, budget), np.float32)
    for i in range(b):
        n = min(max(int(lens[i]), 0), width * page)
        blocks = -(-n // page)
        there = [j for j in range(blocks) if table[i, j] >= 0 or j == blocks - 1]
        total = weights[i].astype(np.float64).sum(0)
        rank = lambda j: (0 if np.isnan(total[j]) else 1, -total[j] if not np.isnan(total[j]) else 0.0, j)  # noqa: E731
        last = sorted((j for j in there if j >= blocks - recent), reverse=True)
        first = sorted(j for j in there if j < blocks - recent and j < sink)
        rest = sorted((j for j in there if j < blocks - recent and j >= sink), key=rank)
        keep = sorted((last + first + rest)[:budget])
        out[i, :len(keep)] = table[i, keep]
        moved[i][:, :len(keep)] = weights[i][:, keep]
        gone = [table[i, j] for j in there if j not in set(keep) and table[i, j] >= 0]
        freed[i, :len(gone)] = gone
        if keep:
            tokens[i] = (len(keep) - 1) * page + (n - 1) % page + 1
    return out, tokens, freed, moved
