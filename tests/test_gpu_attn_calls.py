"""GPU: what the attention side's calls do with arguments that go together, or do not."""
import warnings

import pytest
import torch

from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prepared", [False, True])
def test_positions_without_a_table(prepared):
    """Keys are stored as they are, and the caller is warned, at the line of the call; with neither nothing is said."""
    dev = device()
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device=dev)
    k = torch.randn(3, 1, 64, device=dev).to(torch.bfloat16)
    slots, pos = torch.arange(3, device=dev), torch.arange(5, 8, dtype=torch.int32, device=dev)
    with pytest.warns(UserWarning, match="rotary table") as seen:
        if prepared:
            B.kv_append_prepared(cache, k, k, slots, positions=pos)()
        else:
            B.kv_append(cache, k, k, slots, positions=pos)
    assert [w.filename for w in seen] == [__file__]
    assert torch.equal(B.kv_read(cache, slots)[0], k)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        B.kv_append(cache, k, k, slots)
        B.kv_append(cache, k, k, slots, positions=pos, table=B.rope_table(64, device=dev))
