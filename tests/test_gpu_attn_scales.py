"""GPU parity: attention with tensor scales, softmax scales and queries near the ends of their ranges."""
import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B
from helpers import device
from test_gpu_attn_decode import FORMATS, IDS, Batch

pytestmark = pytest.mark.gpu


def scaled(dev, fmt, k_scale=1.0, v_scale=1.0, size=1.0, seed=0):
    """A Batch whose keys, values and queries have the sizes k_scale, v_scale and `size`."""
    x = Batch(dev, fmt, [333, 20, 0, 1], 6, 2, 128, 64, seed=seed, scales=(k_scale, v_scale) if fmt == 2 else (1.0, 1.0))
    rng = np.random.default_rng(seed + 1)
    n = sum(x.lens)
    k, v = (torch.from_numpy((rng.standard_normal((n, 2, 128)) * s).astype(np.float32)) for s in (k_scale, v_scale))
    user = np.repeat(np.arange(4), x.lens)
    j = np.concatenate([np.arange(m) for m in x.lens])
    slots = x.table.cpu().long()[user, j // 64] * 64 + torch.from_numpy(j % 64)
    B.kv_append(x.cache, k.to(dev), v.to(dev), slots.to(dev))
    x.k, x.v = R.stored(k.numpy(), fmt, x.scales[0]), R.stored(v.numpy(), fmt, x.scales[1])
    x.q = (x.q.float() * size).to(torch.bfloat16)
    assert np.abs(x.k).max() > k_scale and np.abs(x.v).max() > v_scale and x.q.abs().max() > size
    return x


@pytest.mark.parametrize("k_scale", [2.0 ** -64, 2.0 ** -40, 0.3, 2.0 ** 40, 2.0 ** 64])
@pytest.mark.parametrize("v_scale", [2.0 ** -64, 1.7, 2.0 ** 64])
def test_tensor_scales(k_scale, v_scale):
    dev = device()
    x = scaled(dev, B.NVFP4_KV_NVFP4, k_scale, v_scale)
    scale = 1 / (k_scale * 11)
    x.check(*x.call(scale=scale), scale=float(np.float32(scale)))


@pytest.mark.parametrize("fmt,size,k_scale", [
    (0, 2.0 ** -126, 1.0), (0, 2.0 ** 120, 1.0), (1, 2.0 ** -126, 1.0), (1, 2.0 ** 120, 1.0),
    (2, 2.0 ** -96, 1.0), (2, 2.0 ** -112, 1.0), (2, 2.0 ** -120, 1.0), (2, 2.0 ** -126, 2.0 ** 30), (2, 2.0 ** -130, 2.0 ** 64),
    (2, 2.0 ** -64, 2.0 ** -56), (2, 2.0 ** -40, 2.0 ** 64), (2, 2.0 ** 60, 2.0 ** 60), (2, 2.0 ** 120, 1.0),
    (2, 2.0 ** 120, 2.0 ** -64), (2, 2.0 ** -10, 2.0 ** -64)])
def test_query_sizes(fmt, size, k_scale):
    """Queries of any size (below 2^-126 they keep fewer bits themselves) with a softmax scale that makes scores of about one,
    whatever intermediate products of the scales would be."""
    dev = device()
    x = scaled(dev, fmt, k_scale, 1.0, size, seed=3)
    scale = float(np.float32(2.0 ** -4 / size / k_scale))
    x.check(*x.call(scale=scale), scale=scale)
