"""GPU parity: the key-value cache at the ends of its formats' ranges."""
import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu

FP32_MAX = float(np.finfo(np.float32).max)
BF16_MAX = float(torch.finfo(torch.bfloat16).max)
E4M3_MAX = 1.875 * 2.0 ** 127      # code 240 under 2^120


@pytest.mark.parametrize("top", [3.0e38, 247 * 2.0 ** 120, 248 * 2.0 ** 120, 249 * 2.0 ** 120, BF16_MAX, FP32_MAX])
@pytest.mark.parametrize("d", [16, 80, 128, 192, 256])
def test_e4m3_rows_up_to_the_largest_value(top, d):
    """Rows whose maximum is anywhere up to fp32's stay finite: a code for 2^128 saturates at 1.875 * 2^127, within half a step
    (2^-4) of every value there; all other codes by the rule; attention of one token gives its value."""
    dev = device()
    rng = np.random.default_rng(d)
    x = (rng.standard_normal((20, 2, d)) * 2.0 ** 124).astype(np.float32)
    x[:, 0, 3], x[::2, 1, d - 1], x[:, 1, 0] = top, -top, 0.97 * top
    x[5] = top
    cache = B.KvCache(2, 16, 2, d, B.NVFP4_KV_E4M3, device=dev)
    slots = torch.arange(20, device=dev)
    t = torch.from_numpy(x).to(dev)
    B.kv_append(cache, t, t, slots)
    want = np.clip(R.stored(x, B.NVFP4_KV_E4M3), -E4M3_MAX, E4M3_MAX)
    assert (np.abs(want - x.astype(np.float64)) <= 2.0 ** -4 * np.abs(x) + 2.0 ** 110).all()
    for got in B.kv_read(cache, slots, dtype=torch.float32):
        assert np.array_equal(got.double().cpu().numpy(), want)
    q = torch.zeros(20, 2, d, dtype=torch.bfloat16, device=dev)
    table = (slots // 16).int()[:, None].contiguous()
    first = torch.tensor([0, 16], device=dev)
    out = B.attn_decode(q[:2], cache, table[first].contiguous(), torch.ones(2, dtype=torch.int32, device=dev))
    assert np.array_equal(out.double().cpu().numpy(), torch.from_numpy(want[[0, 16]]).to(torch.bfloat16).double().numpy())
