"""The shares that attn_weigh() gives to pages, at scores of any size.

A row's share of a page is sum p_j / l over terms p_j = 2^(s_j - r): whatever the scores' own rounding is, terms enter the
page's sum and l alike, so that the shares of a row add up to 1.  What is left are roundings of positive numbers, each at most
u = 2^-24 of what it rounds: up to n additions into l and moves of its reference (n: the row's tokens; in a lane, eight
additions and one move of four steps at most for 32 of them), sixteen into a sixteen's sum and one for each
sixteen of the page; up to eight steps for each of the two exponentials by which a term's stretch reaches its row's reference
(an exponent d is off by u |d|, which moves 2^-|d| by less than u of the row), and the quotient.  So
(n + 64 + page / 16) u of a row."""
import numpy as np
import pytest
import torch

import attn_reference as R
import long_reference as G
from bit_quantized_decode_amd import binding as B
from test_gpu_kv_evict import Weighed

pytestmark = pytest.mark.gpu


def off(n, page):
    return (n + 64 + page // 16) * R.U24


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("shift", [0, 10, 15, 20, 60, 100])
def test_shares_add_up(fmt, shift):
    """Random scores of every size; rows cut over wavefronts and workgroups, several rows a kv head, a window."""
    for lens, hq, hk, page, window in (([700, 33, 1], 4, 4, 16, 0), ([20000], 2, 1, 64, 0), ([9000, 4000], 6, 2, 64, 5000)):
        x = Weighed(fmt, lens, hq, hk, 64, page, seed=shift + hq)
        w = torch.empty(x.w.shape, device=x.dev)
        _, lse, w = B.attn_weigh(*x.args(), None, 0.0, w, scale=2.0 ** shift / 8, window=window, lse=True)
        assert lse.isfinite().all() and (w >= 0).all()
        w = w.double().sum(-1).cpu().numpy()
        n = np.array([min(n, window) if window else n for n in lens])[:, None]
        err = np.abs(w - hq // hk)
        assert (err <= hq // hk * off(n, page)).all(), (lens, (err / off(n, page)).max())


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("shift", [14, 20, 24, 32, 90])
def test_equal_largest_scores_share(fmt, shift):
    """Some pages hold the row's largest score, several times each, the same number wherever it stands: they share by count, and
    pages without it have nothing.  Both signs of lse, large and small."""
    n, page = 3000, 32
    x = Weighed(fmt, [n], 4, 2, 64, page, seed=shift)
    rng = np.random.default_rng(shift)
    best = np.zeros(n, bool)
    best[rng.choice(n, 37, replace=False)] = True
    best[5 * page:6 * page] = True
    for sign in (1.0, -1.0):
        k = torch.zeros(n, 2, 64)
        k[:, :, 0] = torch.from_numpy(np.where(best, 6.0, 4.0) if sign > 0 else np.where(best, 4.0, 6.0))[:, None]
        x.pool.write(x.pool.slots(x.table[0], n)[0], k.to(torch.bfloat16), torch.ones(n, 2, 64, dtype=torch.bfloat16))
        x.q.zero_()
        x.q[:, :, 0] = sign
        w = torch.empty(x.w.shape, device=x.dev)
        out, lse, w = B.attn_weigh(*x.args(), None, 0.0, w, scale=2.0 ** shift, lse=True)
        count = np.bincount(np.arange(n)[best] // page, minlength=x.w.shape[2])
        want = 2 * count / best.sum()
        err = np.abs(w[0].double().cpu().numpy() - want)
        assert (err <= want * off(n, page)).all(), (sign, err.max())


def test_shares_of_a_row_in_many_parts():
    """One long row with a far score in its last token but one: all earlier pages drop to nothing at once."""
    n, page = 50001, 64
    x = Weighed(B.NVFP4_KV_BF16, [n], 2, 2, 64, page, seed=3)
    k = torch.full((1, 2, 64), 1.0, dtype=torch.bfloat16)
    x.q[:] = 1.0
    at = np.array([x.table[0, (n - 2) // page] * page + (n - 2) % page])
    x.pool.write(at, k * 128, k)
    w = torch.empty(x.w.shape, device=x.dev)
    _, _, w = B.attn_weigh(*x.args(), None, 0.0, w, scale=64.0, lse=True)
    w = w[0].cpu().numpy()
    assert (w[:, :-1] == 0).all() and np.abs(w[:, -1] - 1).max() <= off(n, page)


@pytest.mark.parametrize("fmt", G.FORMATS, ids=G.IDS)
@pytest.mark.parametrize("d", [128, 256])
def test_products_that_cancel(fmt, d):
    """Scores that are small sums of large products: a score is off by up to e = (d + 4) u scale sum |q k|, however small it is, a
    share p_j by p_j (exp(e_j + max e) - 1) from its own and the others' scores, and beyond that by off()."""
    n, page, scale = 50, 16, 0.5
    x = Weighed(fmt, [n], 3, 1, d, page, seed=d)
    rng = np.random.default_rng(d)
    # Channels c and c + d / 8 of each quarter have the same query and opposite keys, but where the query is small.
    pair = lambda a, sign: np.concatenate((a, sign * a), -1).reshape(*a.shape[:-2], d)  # noqa: E731
    k = pair(rng.uniform(0.5, 4, size=(n, 1, 4, d // 8)), -1)
    q = pair(2.0 ** rng.uniform(-6, 6, size=(3, 4, d // 8)), 1)
    q = np.where((q < 0.25) & (np.arange(d) % (d // 4) < d // 8), 0, q)
    x.pool.write(x.pool.slots(x.table[0], n)[0], torch.from_numpy(k.astype(np.float32)).to(torch.bfloat16), torch.ones(n, 1, d, dtype=torch.bfloat16))
    x.q[0] = torch.from_numpy(q).to(torch.bfloat16)
    w = torch.empty(x.w.shape, device=x.dev)
    _, lse, w = B.attn_weigh(*x.args(), None, 0.0, w, scale=scale, lse=True)
    k, q = x.pool.k[x.pool.slots(x.table[0], n)[0], 0], x.q[0].double().numpy()
    s, size = scale * q @ k.T, scale * np.abs(q) @ np.abs(k).T
    assert np.abs(s).max() < 20 and size.min() > 200      # (products do cancel)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    e = (d + 4) * R.U24 * size
    want, bound = (np.add.reduceat(a.sum(0), np.arange(0, n, page)) for a in (p, p * np.expm1(e + e.max(1, keepdims=True))))
    err = np.abs(w[0, 0].double().cpu().numpy() - want)
    assert (err <= bound + 3 * off(n, page)).all(), (err / bound).max()
