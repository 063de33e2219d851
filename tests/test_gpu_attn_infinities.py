"""GPU parity: infinities and NaN in queries, keys and values act as in the formulas, and nowhere else."""
import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B
from helpers import device
from test_gpu_attn_decode import FORMATS, IDS, Batch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
AT = 5          # the element that is not finite


def rewrite(x, b, j, k=None, v=None):
    """Writes token j of sequence b again, with k and v [hk][d] (float32) in place of what it held."""
    start = sum(x.lens[:b]) + j
    slot = (x.table[b, j // x.page].long() * x.page + j % x.page).view(1)
    k = torch.from_numpy(x.k[start]).float() if k is None else k
    v = torch.from_numpy(x.v[start]).float() if v is None else v
    B.kv_append(x.cache, k[None].to(x.dev), v[None].to(x.dev), slot)
    x.k[start], x.v[start] = R.stored(k.numpy(), x.fmt), R.stored(v.numpy(), x.fmt)


def check_head(x, out, lse, b, h, tokens, columns=slice(None)):
    """Query head h of sequence b against the definition over the given tokens."""
    start, kv = sum(x.lens[:b]), h // (x.hq // x.hk)
    k, v = x.k[start:start + x.lens[b]][tokens, kv], x.v[start:start + x.lens[b]][tokens, kv][:, columns]
    o, l, pv, size = R.attend(x.q[b, h:h + 1].double().numpy(), k, v, x.d ** -0.5)
    bo, bl = R.attend_bounds(size, len(k), x.d, o, pv, l, x.fmt, v)
    assert (np.abs(out[b, h:h + 1, columns].double().cpu().numpy() - o) <= bo).all(), (b, h)
    assert (np.abs(lse[b, h:h + 1].double().cpu().numpy() - l) <= bl).all(), (b, h)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_keys(sign):
    """bf16 (other formats hold NaN for an infinite key): against queries of either sign and zero."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_BF16, [200, 40], 8, 2, 64, 32, seed=3)
    x.q[0, :4, AT] = torch.tensor([-1.0, 1.0, 0.0, -0.5])
    key = torch.randn(2, 64, generator=torch.Generator().manual_seed(1)).bfloat16().float()
    key[0, AT] = sign * INF
    rewrite(x, 0, 77, k=key)
    out, lse = x.call()
    others = np.delete(np.arange(200), 77)
    for h in range(4):
        score = float(x.q[0, h, AT]) * sign
        if score < 0:       # a score of -inf: the token weighs nothing
            check_head(x, out, lse, 0, h, others)
        else:               # +inf, or zero times infinity
            assert out[0, h].isnan().all() and lse[0, h].isnan(), h
    for b, h in [(0, 4), (0, 7), (1, 0), (1, 7)]:
        check_head(x, out, lse, b, h, np.arange(x.lens[b]))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_queries(fmt, bad):
    """A query that is not finite concerns its own row alone; keys of one sign beside an infinity give scores of one sign."""
    dev = device()
    x = Batch(dev, fmt, [200, 40], 8, 2, 64, 32, seed=4)
    for b, j in [(b, j) for b, n in enumerate(x.lens) for j in range(n)]:
        start = sum(x.lens[:b]) + j
        key = torch.from_numpy(x.k[start]).float()
        key[:, AT] = -4.0 if b else key[:, AT]
        if b:
            rewrite(x, b, j, k=key)
    x.q[0, 2, AT], x.q[1, 6, AT] = bad, bad
    out, lse = x.call()
    assert out[0, 2].isnan().all() and lse[0, 2].isnan()            # keys of both signs: some score is +inf or NaN
    if bad == INF:                                                  # keys below zero throughout: all scores -inf
        assert (out[1, 6] == 0).all() and lse[1, 6] == -INF
    else:
        assert out[1, 6].isnan().all() and lse[1, 6].isnan()
    for b in range(2):
        for h in range(8):
            if (b, h) not in ((0, 2), (1, 6)):
                check_head(x, out, lse, b, h, np.arange(x.lens[b]))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_values(fmt, bad):
    """A value that is not finite reaches the outputs that hold it (its element, in E4M3 its row, in NVFP4 its block of 16)."""
    dev = device()
    x = Batch(dev, fmt, [200, 40], 8, 2, 64, 32, seed=5)
    value = torch.randn(2, 64, generator=torch.Generator().manual_seed(2)).bfloat16().float()
    value[1, AT] = bad
    rewrite(x, 0, 120, v=value)
    out, lse = x.call()
    hit = {0: slice(AT, AT + 1), 1: slice(0, 64), 2: slice(0, 16)}[fmt]
    rest = {0: slice(AT + 1, 64), 1: slice(0, 0), 2: slice(16, 64)}[fmt]
    for h in range(8):
        if h >= 4:
            assert not out[0, h, hit].isfinite().any(), h
            check_head(x, out, lse, 0, h, np.arange(200), rest)
        else:
            check_head(x, out, lse, 0, h, np.arange(200))
        check_head(x, out, lse, 1, h, np.arange(40))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_outside_a_row_nothing_acts(fmt):
    """Infinities and NaN in tokens before the window, behind the length and in pages that are gone."""
    dev = device()
    x = Batch(dev, fmt, [200], 4, 2, 64, 32, seed=6)
    good = [(torch.from_numpy(x.k[j]).float(), torch.from_numpy(x.v[j]).float()) for j in range(200)]
    for j in (3, 49, 100, 127, 190, 199):
        row = torch.full((2, 64), (INF, NAN, -INF)[j % 3])
        rewrite(x, 0, j, k=row, v=row)
    for j in range(200):
        x.k[j], x.v[j] = (R.stored(t.numpy(), fmt) for t in good[j])
    x.seq = torch.tensor([190], dtype=torch.int32, device=dev)
    x.table[0, 3] = -1                       # tokens 96 .. 127
    out, lse = x.call(window=140)            # tokens 50 .. 189
    tokens = np.concatenate([np.arange(50, 96), np.arange(128, 190)])
    for h in range(4):
        check_head(x, out, lse, 0, h, tokens)
