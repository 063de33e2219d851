"""GPU parity: attention's stated precision and range, each at the edge of what the header promises."""
import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu

FORMATS = [B.NVFP4_KV_BF16, B.NVFP4_KV_E4M3, B.NVFP4_KV_NVFP4]
IDS = ["bf16", "e4m3", "nvfp4"]
HEAD = 64


def one_sequence(dev, fmt, k, v, page=64, scales=(1.0, 1.0)):
    """A cache of one kv head that holds k and v [n][HEAD] (float32) in order, and its page table."""
    n = k.shape[0]
    pages = -(-n // page)
    cache = B.KvCache(pages, page, 1, k.shape[1], fmt, *scales, device=dev)
    cache.pool.fill_(0xff)
    B.kv_append(cache, k[:, None].to(dev), v[:, None].to(dev), torch.arange(n, device=dev))
    return cache, torch.arange(pages, dtype=torch.int32, device=dev)[None]


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_rounding_of_a_weight(fmt):
    """Two tokens whose terms all but cancel, p (-6) and 3 with p about 1/2: what is left shows the rounding of p.

    A term enters the matrix cores within 2^-17 of itself, NVFP4's within 2^-11 (half a step of f16 at the lower end of
    a power of two); all values, weights of the larger token and products are exact.  Besides: p itself, d + 4 half steps of its
    score and four of the exponential, in numerator and sum; and the output's rounding."""
    dev = device()
    k, v = torch.zeros(2, HEAD), torch.full((2, HEAD), 3.0)
    k[1, 0], v[1] = 6.0, -6.0
    cache, table = one_sequence(dev, fmt, k, v)
    q = torch.zeros(1, 1, HEAD, dtype=torch.bfloat16, device=dev)
    q[0, 0, 0] = -1.0
    length = torch.tensor([2], dtype=torch.int32, device=dev)
    weight = 2.0 ** -11 if fmt == B.NVFP4_KV_NVFP4 else 2.0 ** -17
    for j in range(-32, 33):
        scale = float(np.float32(-np.log(0.5 * (1 + j * 2.0 ** -13)) / 6))
        p = np.exp(-6 * scale)
        o = (3 - 6 * p) / (1 + p)
        bound = weight * 6 * p / (1 + p) + ((HEAD + 4) * 6 * scale + 8) * R.U24 * 2 * (3 + 6 * p) / (1 + p) + 2.0 ** -8 * abs(o)
        got = B.attn_decode(q, cache, table, length, scale=scale)[0, 0].double().cpu().numpy()
        assert (np.abs(got - o) <= bound).all(), (j, got[0], o, bound)


@pytest.mark.parametrize("fmt", FORMATS[:2], ids=IDS[:2])
@pytest.mark.parametrize("rise", [0.0, 7.9, 300.0])
def test_largest_values(fmt, rise):
    """Values of 2^127 / n, the first 32 of n tokens `rise` (in base 2) below the others: sums of n terms stay finite.

    As many sequences as fill the GPU, so that a wavefront takes a whole one and meets the rise inside its run.  All weights add up
    to one: each output is its column's value, within its rounding, the terms' and those of two sums of n."""
    dev = device()
    n, b = 512, 2048
    m = 2.0 ** 127 / n
    k, v = torch.zeros(n, HEAD), torch.full((n, HEAD), m)
    k[32:, 0] = 1.0
    v[:, 1::2] = -m / 2
    cache, table = one_sequence(dev, fmt, k, v)
    q = torch.zeros(b, 1, HEAD, dtype=torch.bfloat16, device=dev)
    q[:, 0, 0] = 1.0
    scale = float(np.float32(max(rise, 1e-6) * np.log(2)))
    out, lse = B.attn_decode(q, cache, table.expand(b, -1).contiguous(), torch.full((b,), n, dtype=torch.int32, device=dev),
                             scale=scale, lse=True)
    want = v[0].double().numpy()
    err = np.abs(out[:, 0].double().cpu().numpy() - want)
    assert (err <= (2.0 ** -8 + 2 * (2.0 ** -17 + (n + 8) * R.U24)) * np.abs(want)).all(), err.max() / m
    exact = scale + np.log(n - 32 + 32 * np.exp(-scale))
    assert (np.abs(lse.double().cpu().numpy() - exact) <= (n + 16) * R.U24 * (1 + exact)).all()


@pytest.mark.parametrize("fmt", FORMATS[:2], ids=IDS[:2])
@pytest.mark.parametrize("n", [1, 3])
def test_smallest_values(fmt, n):
    """Values down to the formats' smallest normal ones (2^-126, and 2^-119 of E4M3), equal for all tokens: products with terms
    of 2^-8 and more keep 15 bits below 2^-126, which leaves each output within a step of bf16."""
    dev = device()
    small = 2.0 ** -126 if fmt == B.NVFP4_KV_BF16 else 2.0 ** -119
    v = (torch.arange(1, HEAD + 1) % 2 + 1.0).mul(small).expand(n, HEAD).contiguous()
    cache, table = one_sequence(dev, fmt, torch.zeros(n, HEAD), v)
    out = B.attn_decode(torch.ones(1, 1, HEAD, dtype=torch.bfloat16, device=dev), cache, table,
                        torch.tensor([n], dtype=torch.int32, device=dev))
    want = v[0].double().numpy()
    assert (np.abs(out[0, 0].double().cpu().numpy() - want) <= 2.0 ** -7 * want).all()
