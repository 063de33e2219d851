"""GPU: the attention side's calls at the largest and smallest sizes that the header allows."""
import math

import pytest
import torch

from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu

FORMATS = [B.NVFP4_KV_BF16, B.NVFP4_KV_E4M3, B.NVFP4_KV_NVFP4]
IDS = ["bf16", "e4m3", "nvfp4"]


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("short", [0, 5])
def test_longest_sequence(fmt, short):
    """2^30 tokens, the same page 16,384 times: equal scores and values of small whole numbers, whose sums of equal powers of
    two times those are exact in fp32, so that the output is the mean to bf16's rounding and lse = ln n."""
    dev = device()
    page, times, d = 65536, 16384, 64
    cache = B.KvCache(1, page, 1, d, fmt, device=dev)
    values = torch.tensor([2.0, 4.0, 4.0, 6.0])
    v = values.repeat(page // 4)[:, None, None].expand(page, 1, d).contiguous()
    v[..., ::16] = 6.0          # the largest of each block of 16: its scale is 1, and the others are E2M1 numbers
    k = torch.zeros(page, 1, d)
    B.kv_append(cache, k.to(dev), v.to(dev), torch.arange(page, device=dev))
    n = page * times - short
    q = torch.ones(1, 1, d, dtype=torch.bfloat16, device=dev)
    out, lse = B.attn_decode(q, cache, torch.zeros(1, times, dtype=torch.int32, device=dev),
                             torch.tensor([n], dtype=torch.int32, device=dev), lse=True)
    left_out = v[page - short:].double().sum(0)[None]
    mean = (v.double().sum(0)[None] * times - left_out) / n
    assert ((out.double().cpu() - mean).abs() <= 2.0 ** -8 * mean).all()
    assert abs(float(lse) - math.log(n)) <= 2.0 ** -21 * math.log(n)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_most_rows_of_a_cache_call(fmt):
    """2^24 tokens in one call, written, read back and turned; values on every format's grid come back as they are."""
    dev = device()
    tokens, d = 1 << 24, 16
    cache = B.KvCache(256, 65536, 1, d, fmt, device=dev)
    gen = torch.Generator(device=dev).manual_seed(fmt)
    grid = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=dev).to(torch.bfloat16)
    k = grid[torch.randint(0, 14, (tokens, 1, d), generator=gen, device=dev)]
    k[..., 7] = 6.0
    v = -k
    slots = torch.randperm(tokens, generator=gen, device=dev)
    B.kv_append(cache, k, v, slots)
    k2, v2 = B.kv_read(cache, slots)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    if fmt == B.NVFP4_KV_BF16:
        table = B.rope_table(d, device=dev)
        pos = torch.zeros(tokens, dtype=torch.int32, device=dev)
        pos[-1] = 12345
        y = B.rope(k, pos, table)
        assert torch.equal(y[:-1], k[:-1]) and torch.equal(y[-1:], B.rope(k[-1:], pos[-1:], table))
        assert not torch.equal(y[-1:], k[-1:])


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_no_pages_and_no_sequences(fmt):
    """A table without columns leaves every row empty, whatever its length says; no rows at all is a no-op."""
    dev = device()
    cache = B.KvCache(1, 16, 2, 64, fmt, device=dev)
    cache.pool.fill_(0xff)
    q = torch.randn(3, 4, 64, device=dev).to(torch.bfloat16)
    lens = torch.tensor([0, 7, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    for call in (B.attn_decode, lambda *a, **kw: B.attn_decode_prepared(*a, **kw)()):
        out, lse = call(q, cache, torch.empty(3, 0, dtype=torch.int32, device=dev), lens, lse=True, window=3)
        assert (out == 0).all() and torch.isneginf(lse).all()
        out, lse = call(q[:0], cache, torch.empty(0, 5, dtype=torch.int32, device=dev), lens[:0], lse=True)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
